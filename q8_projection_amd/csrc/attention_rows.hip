// attention_rows.hip -- attention of many rows a sequence and kv head (prompts, chunks of prompts, drafts
// of large groups): bound by the matrix cores.
//
// A workgroup of 4 waves takes a tile of 64 NR query rows of one sequence and kv head (a token's query heads
// side by side), 16 NR a wave, and walks over the tokens that they see.  Keys and values become binary16
// once for the workgroup: each wave turns a quarter of the next tokens' codes into operands of the matrix
// cores and leaves them in LDS, in the order in which a wave takes them (no bank conflicts), while all
// multiply the present ones; one barrier a step.  Two workgroups a CU, so that one's softmax runs beside
// the other's products.
//
// Row tiles of causal prompts differ in length: the longest come first, and every second round over the
// CUs in the other order, so that what one CU gets together is about even.  Few row tiles are divided over the
// tokens into pieces, joined by the last workgroup to finish one, in the pieces' order.
#include <algorithm>

#include "attention.h"
#include "launch.h"

namespace q8 {
namespace {

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kPerCu = 2;
static_assert(2 * kPerCu <= kCountersPerCu);
constexpr int kMinTiles = 16;  // tiles of a piece, at least (but for shorter spans)

// Rows of a lane column: 32 rows a wave are 128 registers of queries and sums (D = 128); 256 dimensions
// leave room for 16.
template <int D>
constexpr int kRowTiles = D == 256 ? 1 : 2;

struct RowsArgs {
    AttentionArgs a;
    int cus;
    int pieces;         // wanted
    uint32_t *arrived;  // [2 pieces], zero between calls
    float *parts;       // [2 pieces][slot]
};

// Floats of a part: sums of a row tile, then (maximum, sum) of its rows.
constexpr int slot_of(int d) { return (d == 256 ? 64 : 128) * (d + 4); }

// The rows of tile `x` of a sequence's rows.
__device__ __forceinline__ Rows rows_of_tile(const AttentionArgs &a, const Rows &r, int x, int tile_rows) {
    const int from = x * tile_rows / a.group, to = min((x + 1) * tile_rows + a.group - 1, r.n * a.group) / a.group;
    return {r.first + from, to - from, r.at + from, r.end};
}

struct Piece {
    int s, tile, head, index, n;
    int64_t first;  // its row tile's first part
    Rows rows;      // of the sequence
};

// Finds pieces by their place in the order of sequences, row tiles (last first), parts and heads.
template <int TILE>
struct Pieces {
    int target;  // tiles of 32 tokens of a piece at most
    int s0 = 0;
    int64_t pieces = 0, parts = 0;
    Rows rows;
    uint32_t tiles, count, scan, scan_parts;  // row tiles, pieces of each

    // Row tiles times the tiles of tokens that the last one sees (the longest).
    __device__ __forceinline__ int64_t look(const AttentionArgs &a, int lane) {
        const int s = s0 + lane;
        rows = Rows{0, 0, 0, 0};
        if (s < a.c.sequences) rows = sequence_rows(a.c, s);
        tiles = (static_cast<uint32_t>(rows.n) * a.group + TILE - 1) / TILE;
        if (!tiles) return 0;
        return int64_t(tiles) * last(a);
    }
    __device__ __forceinline__ int last(const AttentionArgs &a) const {
        return span_of(a, rows_of_tile(a, rows, static_cast<int>(tiles) - 1, TILE)).n;
    }
    __device__ __forceinline__ void divide(const AttentionArgs &a) {
        count = tiles ? static_cast<uint32_t>((last(a) + target - 1) / target) : 0u;
        scan = wave_scan(tiles * count);
        scan_parts = wave_scan(count > 1 ? tiles * count : 0u);
    }
    __device__ __forceinline__ void rewind(const AttentionArgs &a, int lane) {
        if (s0 == 0 && pieces == 0) return;
        s0 = 0;
        pieces = parts = 0;
        look(a, lane);
        divide(a);
    }
    __device__ __forceinline__ bool find(const AttentionArgs &a, int64_t p, int lane, Piece &out) {
        if (p < pieces) rewind(a, lane);
        for (;;) {
            const uint64_t above = __ballot(pieces + int64_t(scan) * a.c.kv_heads > p);
            if (above) {
                const int l = __builtin_ctzll(above);
                const int64_t before = pieces + (l ? int64_t(lane_of(scan, l - 1)) * a.c.kv_heads : 0);
                const int n = static_cast<int>(lane_of(count, l)), rest = static_cast<int>(p - before);
                out.s = s0 + l;
                out.n = n;
                out.head = rest % a.c.kv_heads;
                const int x = rest / a.c.kv_heads;
                out.index = x % n;
                out.tile = static_cast<int>(lane_of(tiles, l)) - 1 - x / n;
                out.first = parts + (l ? int64_t(lane_of(scan_parts, l - 1)) * a.c.kv_heads : 0) +
                            (int64_t(out.tile) * a.c.kv_heads + out.head) * n;
                out.rows = Rows{static_cast<int>(lane_of(rows.first, l)), static_cast<int>(lane_of(rows.n, l)),
                                static_cast<int>(lane_of(rows.at, l)), static_cast<int>(lane_of(rows.end, l))};
                return true;
            }
            if (s0 + 64 >= a.c.sequences) return false;
            pieces += int64_t(lane_of(scan, 63)) * a.c.kv_heads;
            parts += int64_t(lane_of(scan_parts, 63)) * a.c.kv_heads;
            s0 += 64;
            look(a, lane);
            divide(a);
        }
    }
};

// What a wave turns into operands in one step of kStep tokens: a quarter of the codes.
template <int BITS, int D>
struct Codes {
    using T = Tile<BITS, D>;
    using O = Out<BITS, D>;
    static constexpr int kStep = 8192 / D;                                // tokens: 32 KB of operands
    static constexpr int kUnits = BITS == 4 ? (D + 127) / 128 : D / 64;   // loads of a token's keys
    static constexpr int kIn = BITS == 4 ? (D == 64 ? 2 : 4) : 2;         // operands of a load
    static constexpr int kKeys = kStep / 16 * kUnits / kWaves, kValues = kStep / 32 * O::kChunks / kWaves;

    u32x4 k[kKeys], v[kValues], vw[kValues][O::kBlocks];
    uint32_t kw[kKeys];

    // tile_of(i): the i-th tile of the step
    template <typename Fn>
    __device__ __forceinline__ void load(Fn tile_of, int wid, uint32_t g, uint32_t c) {
        const uint32_t t = (c >> 2) * 8 + (c & 3);
        const uint32_t code = t * T::kRow + g * (BITS == 4 && D == 64 ? 8 : 16);
        const uint32_t word = T::kKeyWords + (c * T::kBlocks + (BITS == 4 && D > 64 ? g : g >> 1)) * 4;
        const uint32_t u = O::unit(c);
        const uint32_t vcode = T::kValues + ((u * 4 + g) * 16 + O::chunk(c, 0)) * 16;
        const uint32_t vword = T::kValueWords + (u * O::kBlocks * 4 + g) * 16;
#pragma unroll
        for (int q = 0; q < kKeys; ++q) {
            const int unit = wid + kWaves * q, half = unit / kUnits, part = unit % kUnits;
            const uint8_t *tile = tile_of(half >> 1), *p = tile + 4 * (half & 1) * T::kRow + part * 64;
            if (BITS == 4 && D == 64) {
                const u32x2 x = *reinterpret_cast<const u32x2 *>(p + code);
                k[q] = u32x4{x.x, x.y, 0, 0};
            } else {
                k[q] = *reinterpret_cast<const u32x4 *>(p + code);
            }
            kw[q] = *reinterpret_cast<const uint32_t *>(tile + part * (BITS == 4 ? 16 : 8) + word);
        }
#pragma unroll
        for (int q = 0; q < kValues; ++q) {
            const int unit = wid + kWaves * q;
            const uint8_t *tile = tile_of(unit / O::kChunks);
            v[q] = *reinterpret_cast<const u32x4 *>(tile + unit % O::kChunks * 16 + vcode);
#pragma unroll
            for (int b = 0; b < O::kBlocks; ++b) vw[q][b] = *reinterpret_cast<const u32x4 *>(tile + b * 64 + vword);
        }
    }

    // Operands to LDS: keys [half][step][lane], values [tile][operand][lane].  there(i, p): the halves of
    // a word pair whose tokens (p, p + 4 of the lane's eight) of the step's tile i are there.
    template <typename Fn>
    __device__ __forceinline__ void store(half8 *keys, half8 *values, Fn there, int wid, int lane) const {
#pragma unroll
        for (int q = 0; q < kKeys; ++q) {
            const int unit = wid + kWaves * q, half = unit / kUnits, part = unit % kUnits;
            Scales<BITS> sc;
            sc.set(__builtin_amdgcn_perm(kw[q], kw[q], half & 1 ? 0x03020302u : 0x01000100u));
#pragma unroll
            for (int e = 0; e < kIn; ++e) {
                half8 x;
                if constexpr (BITS == 4) x = values_of(k[q][e], sc, sc, sc, sc);
                else x = values_of(k[q][2 * e], k[q][2 * e + 1], sc, sc, sc, sc);
                keys[(half * (D / 32) + part * kIn + e) * 64 + lane] = x;
            }
        }
#pragma unroll
        for (int q = 0; q < kValues; ++q) {
            const int unit = wid + kWaves * q, tile = unit / O::kChunks, m = unit % O::kChunks;
            Scales<BITS> sc[O::kBlocks][4];
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t mask = there(tile, p);
#pragma unroll
                for (int b = 0; b < O::kBlocks; ++b) sc[b][p].set(vw[q][b][p] & mask);
            }
#pragma unroll
            for (int w = 0; w < O::kIn; ++w) {
                half8 x;
                if constexpr (BITS == 4) x = values_of(v[q][w], sc[w / 2][0], sc[w / 2][1], sc[w / 2][2], sc[w / 2][3]);
                else x = values_of(v[q][2 * w], v[q][2 * w + 1], sc[0][0], sc[0][1], sc[0][2], sc[0][3]);
                values[(tile * (D / 16) + m * O::kIn + w) * 64 + lane] = x;
            }
        }
    }
};

template <int BITS, int D>
__global__ __launch_bounds__(kThreads, kPerCu) void rows_kernel(RowsArgs f) {
    using O = Out<BITS, D>;
    using C = Codes<BITS, D>;
    constexpr int NR = kRowTiles<D>, kTile = 64 * NR, kSteps = D / 32, kSlot = slot_of(D);
    constexpr int kTiles = C::kStep / kTileTokens;  // tiles of a step
    __shared__ half8 keys[2][16 * 64], values[2][16 * 64];
    __shared__ uint32_t last;
    const AttentionArgs &a = f.a;
    const CacheArgs &c = a.c;
    const int lane = threadIdx.x & 63, g = lane >> 4, col = lane & 15;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

    Pieces<kTile> pieces;
    int64_t total = 0;
    for (; pieces.s0 < c.sequences; pieces.s0 += 64) {
        int64_t n = pieces.look(a, lane);
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) n += __shfl_xor(n, off, 64);
        total += n;
    }
    // (no span has more than 2^25 tiles)
    pieces.target = static_cast<int>(min(max((total * c.kv_heads + f.pieces - 1) / f.pieces, int64_t(kMinTiles)), int64_t(1) << 26));
    int64_t all = 0;
    for (pieces.s0 = 0; pieces.s0 < c.sequences; pieces.s0 += 64) {
        if (c.sequences > 64) pieces.look(a, lane);
        pieces.divide(a);
        all += int64_t(lane_of(pieces.scan, 63)) * c.kv_heads;
    }
    pieces.s0 = 0;
    if (c.sequences > 64) {
        pieces.look(a, lane);
        pieces.divide(a);
    }

    Piece piece;
    for (int64_t p = blockIdx.x; p < all; p += gridDim.x) {
        // every second round over the CUs backwards
        const int64_t round = p / f.cus, in = p - round * f.cus;
        const int64_t size = min(int64_t(f.cus), all - round * f.cus);
        if (!pieces.find(a, round & 1 ? round * f.cus + size - 1 - in : p, lane, piece)) return;
        const Rows r = piece.rows, tile_rows = rows_of_tile(a, r, piece.tile, kTile);
        const Span span = span_of(a, tile_rows);
        const int from = static_cast<int>(int64_t(span.n) * piece.index / piece.n);
        const int to = static_cast<int>(int64_t(span.n) * (piece.index + 1) / piece.n);
        const int rows = r.n * a.group, row0 = piece.tile * kTile, head = piece.head;
        // tokens that any row of the tile sees, and those that every one does
        const int lo = a.window ? max(tile_rows.at - a.window + 1, 0) : 0, hi = min(tile_rows.at + tile_rows.n, r.end);
        const int all_lo = a.window ? max(tile_rows.at + tile_rows.n - a.window, 0) : 0, all_hi = min(tile_rows.at + 1, r.end);

        // Pages of 64 tiles at a time, one a lane.
        const int shift = c.page_shift - 5;
        int paged = 0, page = -1;
        const auto look_up = [&](int tile) {
            paged = tile;
            const int t = span.first + tile + lane;
            page = -1;
            if (tile + lane < to && t * kTileTokens < hi) page = c.table[piece.s * c.table_ld + (t >> shift)];
            if (page < 0 || page >= c.pages) page = -1;
        };
        const auto page_of = [&](int tile) {  // -1 past the last one
            return tile < to ? __builtin_amdgcn_readlane(page, tile - paged) : -1;
        };
        const auto tile_of = [&](int tile) -> const uint8_t * {
            const int t = span.first + tile;
            const int64_t pg = max(page_of(tile), 0);  // (none: the pool's first, not looked at)
            return c.data + (((pg * c.kv_heads + head) << shift) + (t & ((1 << shift) - 1))) * Tile<BITS, D>::kBytes;
        };

        C codes;
        // Which of a step's tiles are there, as bits, and the load of its codes.
        uint32_t there_next = 0;
        const auto load = [&](int tile) {
            if (tile - paged + kTiles > 64 || tile < paged) look_up(tile);
            there_next = 0;
#pragma unroll
            for (int i = 0; i < kTiles; ++i) there_next |= (page_of(tile + i) >= 0 ? 1u : 0u) << i;
            codes.load([&](int i) { return tile_of(tile + i); }, wid, g, col);
        };
        const auto store = [&](int tile, uint32_t there_bits, int buf) {
            codes.store(keys[buf], values[buf],
                        [&](int i, int pair) {
                            const int t0 = (span.first + tile + i) * kTileTokens;
                            if (!(there_bits >> i & 1)) return 0u;
                            if (t0 >= lo && t0 + kTileTokens <= hi) return 0xffffffffu;
                            const int t = t0 + 8 * g + pair;
                            return (t >= lo && t < hi ? 0xffffu : 0u) | (t + 4 >= lo && t + 4 < hi ? 0xffff0000u : 0u);
                        },
                        wid, lane);
        };

        look_up(from);
        load(from);
        half8 q_hi[NR][kSteps], q_lo[NR][kSteps];
        float to_score[NR], top[NR], sum[NR];
        int begin[NR], end[NR];
        f32x4 acc[NR][O::kChunks][O::kIn];
        // this wave's rows, and the tokens that they see
        const int first_row = row0 + wid * 16 * NR, last_row = min(first_row + 16 * NR, rows) - 1;
        const int wave_end = last_row < first_row ? 0 : min(r.at + last_row / a.group + 1, r.end);
        const int wave_begin = a.window ? max(r.at + first_row / a.group - a.window + 1, 0) : 0;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int x = first_row + n * 16 + col;
            const float *row = nullptr;
            begin[n] = end[n] = 0;
            if (x < rows) {
                const Where q = where(a, r, head, x);
                row = a.q + q.row * a.q_ld + int64_t(q.head) * D;
                const int at = r.at + x / a.group;
                begin[n] = a.window ? max(at - a.window + 1, 0) : 0;
                end[n] = min(at + 1, r.end);
            }
            to_score[n] = load_query<BITS, D>(row, a.scale, g, [&](int s, half8 hi8, half8 lo8) { q_hi[n][s] = hi8, q_lo[n][s] = lo8; });
            top[n] = kNoMax;
            sum[n] = 0.0f;
#pragma unroll
            for (int m = 0; m < O::kChunks; ++m)
#pragma unroll
                for (int j = 0; j < O::kIn; ++j) acc[n][m][j] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        uint32_t there = there_next;
        store(from, there, 0);
        if (from + kTiles < to) load(from + kTiles);
        __syncthreads();
        int buf = 0;
        for (int tile = from; tile < to; tile += kTiles, buf ^= 1) {
            const uint32_t now = there;
            if (tile + kTiles < to) {
                there = there_next;
                store(tile + kTiles, there, buf ^ 1);
                if (tile + 2 * kTiles < to) load(tile + 2 * kTiles);
            }
#pragma unroll
            for (int i = 0; i < kTiles; ++i) {
                const int t0 = (span.first + tile + i) * kTileTokens;
                if (!(now >> i & 1) || t0 >= wave_end || t0 + kTileTokens <= wave_begin) continue;
                const bool masked = t0 < all_lo || t0 + kTileTokens > all_hi;
                f32x4 z[NR][2];
#pragma unroll
                for (int n = 0; n < NR; ++n) z[n][0] = z[n][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int s = 0; s < kSteps; ++s) {
                    const half8 k0 = keys[buf][(2 * i * kSteps + s) * 64 + lane], k1 = keys[buf][((2 * i + 1) * kSteps + s) * 64 + lane];
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        z[n][0] = mfma(k0, q_hi[n][s], z[n][0]);
                        z[n][1] = mfma(k1, q_hi[n][s], z[n][1]);
                    }
#pragma unroll
                    for (int n = 0; n < NR; ++n) {
                        z[n][0] = mfma(k0, q_lo[n][s], z[n][0]);
                        z[n][1] = mfma(k1, q_lo[n][s], z[n][1]);
                    }
                }
                half8 p_hi[NR], p_lo[NR];
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    weigh(z[n], masked, t0, g, begin[n], end[n], to_score[n], top[n], sum[n], acc[n], p_hi[n], p_lo[n]);
#pragma unroll
                for (int m = 0; m < O::kChunks; ++m)
#pragma unroll
                    for (int w = 0; w < O::kIn; ++w) {
                        const half8 v = values[buf][(i * (D / 16) + m * O::kIn + w) * 64 + lane];
#pragma unroll
                        for (int n = 0; n < NR; ++n) acc[n][m][w] = mfma(v, p_hi[n], acc[n][m][w]);
#pragma unroll
                        for (int n = 0; n < NR; ++n) acc[n][m][w] = mfma(v, p_lo[n], acc[n][m][w]);
                    }
            }
            __syncthreads();
        }

        const __amdgpu_buffer_rsrc_t parts = parts_of(f.parts + piece.first * kSlot, piece.n * kSlot);
#pragma unroll
        for (int n = 0; n < NR; ++n) {
            const int x = first_row + n * 16 + col;
            const float total_x = column_sum(sum[n]);
            if (x >= rows) continue;
            const float scale = Scales<BITS>::kUp;
            if (piece.n == 1) {
                const Where at = where(a, r, head, x);
                O::for_each_vec(acc[n], g, [&](int dim, f32x4 v) { write_row<D>(a, at, dim, v * scale, total_x, top[n]); });
            } else {
                const int y = x - row0, slot = piece.index * kSlot;
                O::for_each_vec(acc[n], g, [&](int dim, f32x4 v) { store_part(parts, slot + y * D + dim, v * scale); });
                if (g == 0) store_part(parts, slot + kTile * D + 4 * y, f32x4{top[n], total_x, 0.f, 0.f});
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
                const int vecs = min(rows - row0, kTile) * (D / 4);
                for (int e = threadIdx.x; e < vecs; e += kThreads) {
                    const int y = e / (D / 4), dim = e % (D / 4) * 4;
                    Sums joined;
                    constexpr int kAhead = 4;
                    for (int i = 0; i < piece.n; i += kAhead) {
                        f32x4 o[kAhead], st[kAhead];
#pragma unroll
                        for (int j = 0; j < kAhead; ++j) {
                            // (past the last one: past the buffer, nothing is read)
                            const uint32_t at = static_cast<uint32_t>((i + j) * kSlot) | oob_bit(i + j < piece.n) >> 2;
                            st[j] = load_part(parts, at + kTile * D + 4 * y);
                            o[j] = load_part(parts, at + 4 * e);
                        }
#pragma unroll
                        for (int j = 0; j < kAhead; ++j)
                            if (i + j < piece.n) joined.add(o[j], st[j].x, st[j].y);
                    }
                    write_row<D>(a, where(a, r, head, row0 + y), dim, joined.o, joined.sum, joined.top);
                }
            }
            __syncthreads();  // last is free again
        }
    }
}

int rows_pieces() { return device_info().cus * kPerCu; }

template <int BITS, int D>
hipError_t run(const RowsArgs &f, hipStream_t stream) {
    constexpr int kTile = 64 * kRowTiles<D>;
    const int64_t row_tiles = (int64_t(f.a.c.max_rows) * f.a.group + kTile - 1) / kTile;
    const int64_t most = f.pieces + int64_t(f.a.c.sequences) * f.a.c.kv_heads * row_tiles;
    const dim3 grid(static_cast<uint32_t>(std::min<int64_t>(most, 8 * int64_t(f.pieces))));
    rows_kernel<BITS, D><<<grid, kThreads, 0, stream>>>(f);
    return hipGetLastError();
}

}  // namespace

int64_t rows_workspace(int dim) { return attention_counter_bytes() + int64_t(2) * rows_pieces() * slot_of(dim) * 4; }

hipError_t launch_rows(int bits, int dim, const AttentionArgs &a, void *workspace, hipStream_t stream) {
    RowsArgs f = {};
    f.a = a;
    f.cus = device_info().cus;
    f.pieces = rows_pieces();
    f.arrived = static_cast<uint32_t *>(workspace);
    f.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + attention_counter_bytes());
    if (bits == 4) return dim == 64 ? run<4, 64>(f, stream) : dim == 128 ? run<4, 128>(f, stream) : run<4, 256>(f, stream);
    return dim == 64 ? run<8, 64>(f, stream) : dim == 128 ? run<8, 128>(f, stream) : run<8, 256>(f, stream);
}

}  // namespace q8
