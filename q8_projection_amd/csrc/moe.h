// moe.h -- arguments shared by the kernels of the mixture-of-experts layer, and
// the layout of its workspace.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q8 {

constexpr int kMoeSlice = 64;        // rows one pass serves: a token set fits one 64-bit mask
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeMaxPairs = kMoeSlice * kMoeMaxTopK;

// Counters at the head of the workspace, a cache line each: workgroups that count in on
// one line wait for each other (1024 of them on 16 neighbouring words took 12 us).
constexpr int kMoeCounterStride = 32;  // words
constexpr int kMoeMaxSplits = 8;
constexpr int kMoeTileCounter = 32 * kMoeCounterStride;  // first of the down projection's counters, one a tile
constexpr int kMoeMaxTiles = 512;                        // tiles whose work is split
constexpr int kMoeCounterBytes = (kMoeTileCounter + kMoeMaxTiles) * 4;

// One chosen expert: its tokens are the set bits of `mask` in ascending order,
// and token number i of them is pair `offset + i`.
struct MoeEntry {
    int32_t expert;
    int32_t offset;
    uint64_t mask;
};

// What the plan tells the expert kernels.
struct MoePlan {
    int32_t n_active;
    int32_t pad[3];
    MoeEntry entry[kMoeMaxExperts];
    int32_t pair_token[kMoeMaxPairs];
    double pair_gate[kMoeMaxPairs];
};

struct MoeArgs {
    const float *x;         // [rows][k]
    const float *router;    // [experts][k] or null (choices given)
    const uint8_t *w_gate;  // Q8_0 blocks [experts][ff][nbk]
    const uint8_t *w_up;
    const uint8_t *w_down;  // Q8_0 blocks [experts][k][nbf]
    const float *residual;  // [rows][k] or null
    float *y;               // [rows][k]
    int32_t *ids;           // [rows][top_k] (written by the router, or given)
    float *gates;
    int rows;               // 1 .. 64
    int experts;
    int top_k;
    int renormalize;
    int k, nbk;
    int ff, nbf;
    int tiled;              // on the matrix cores, quantized activations in their order (below)
    int sbk, sbf;           // blocks of one row of xq and hq: nbk and nbf, rounded up to four if tiled
    int splits;             // workgroups that share a tile of the down projection
    // workspace
    double *parts;          // [k / 32][splits][rows][32] partial outputs (splits > 1)
    uint32_t *counters;     // zero between calls
    MoePlan *plan;
    float *logits;          // [rows][experts]
    // Quantized rows.  Plain order: [row][block][word][32].  Tiled: [row][block / 4][word]
    // [part 0..3][block % 4][8]: the four 8-byte parts that one lane of the matrix cores
    // takes of four blocks are 32 bytes in a row; blocks that round a row up are zero.
    uint8_t *xq;            // [rows][sbk] records of words * 32 bytes
    float *xs;              // [rows][sbk]
    uint8_t *hq;            // [pairs][sbf] records (f32 mode: f32 [pairs][ff])
    float *hs;              // [pairs][sbf]
};

// Byte offset of dword `part` (0..7) of block `blk`'s word in its row of records.
__host__ __device__ inline int record_offset(int tiled, int words, int blk, int word, int part) {
    return tiled ? (blk >> 2) * (words * 128) + word * 128 + (part >> 1) * 32 + (blk & 3) * 8 + (part & 1) * 4
                 : blk * (words * 32) + word * 32 + part * 4;
}

// Whether the experts run on the matrix cores: for a mean of more than two tokens an
// expert, in the f32 mode more than three.  Both ways, vector and matrix, in us a layer (64
// experts of which 8 are chosen, k 2048, ff 1408; two words | one word | f32): mean 1: 100, 100 |
// | 161, 257; mean 2: 144, 134 | 132, 141 | 241, 335; mean 3: 168, 148; mean 4: 204, 163 |
// 180, 159 | 386, 372; mean 5: 237, 166; mean 6: | 224, 171 | 535, 383; mean 8: | | 720, 389.
inline int moe_tiled(int words, const MoeArgs &a) { return a.rows * a.top_k > (words ? 2 : 3) * a.experts; }

// Output columns of a workgroup of the down projection on the matrix cores.
constexpr int kMoeDownRows = 32;

// Workgroups that share a tile of them in the down projection on the
// matrix cores: enough for two workgroups a CU.
inline int moe_down_splits(const MoeArgs &a) {
    if (!a.tiled) return 1;
    int s = 1;
    while (s < kMoeMaxSplits && a.k / kMoeDownRows * s < 512) s *= 2;
    return s;
}

inline int64_t moe_align(int64_t v) { return (v + 255) / 256 * 256; }

// Places the workspace's parts (base may be null: sizes only); returns its bytes.
inline int64_t moe_layout(MoeArgs &a, uint8_t *base, int words) {
    const int64_t rows = a.rows, pairs = rows * a.top_k;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        uint8_t *p = base ? base + at : nullptr;
        at += moe_align(bytes);
        return p;
    };
    a.counters = reinterpret_cast<uint32_t *>(take(kMoeCounterBytes));
    a.plan = reinterpret_cast<MoePlan *>(take(sizeof(MoePlan)));
    a.logits = reinterpret_cast<float *>(take(rows * a.experts * 4));
    a.tiled = moe_tiled(words, a);
    a.sbk = a.tiled && words ? (a.nbk + 3) / 4 * 4 : a.nbk;
    a.sbf = a.tiled && words ? (a.nbf + 3) / 4 * 4 : a.nbf;
    a.splits = moe_down_splits(a);
    a.xq = take(rows * a.sbk * words * 32);
    a.xs = reinterpret_cast<float *>(take(words ? rows * a.sbk * 4 : 0));
    a.hq = take(words ? pairs * a.sbf * words * 32 : pairs * a.ff * 4);
    a.hs = reinterpret_cast<float *>(take(words ? pairs * a.sbf * 4 : 0));
    a.parts = reinterpret_cast<double *>(take(a.splits > 1 ? int64_t(8) * a.splits * rows * a.k : 0));
    return at;
}

// mode: 0 f32, 1 one-word, 2 two-word.  route: the router's logits, choices and
// gates; experts: the projections (with the router's choices, or given ones).
hipError_t launch_moe(int mode, const MoeArgs &a, bool route, bool experts, hipStream_t stream);

}  // namespace q8
