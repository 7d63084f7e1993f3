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
    // workspace
    uint32_t *counters;     // zero between calls
    MoePlan *plan;
    float *logits;          // [rows][experts]
    uint8_t *xq;            // [rows][nbk][words * 32]: a block's hi words, then its lo words
    float *xs;              // [rows][nbk]
    uint8_t *hq;            // [pairs][nbf][words * 32] (f32 mode: f32 [pairs][ff])
    float *hs;              // [pairs][nbf]
};

// Counters at the head of the workspace, a cache line each: workgroups that count in on
// one line wait for each other (1024 of them on 16 neighbouring words took 12 us).
constexpr int kMoeCounterStride = 32;  // words
constexpr int kMoeCounterBytes = 32 * kMoeCounterStride * 4;

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
    a.xq = take(rows * a.nbk * words * 32);
    a.xs = reinterpret_cast<float *>(take(words ? rows * a.nbk * 4 : 0));
    a.hq = take(words ? pairs * a.nbf * words * 32 : pairs * a.ff * 4);
    a.hs = reinterpret_cast<float *>(take(words ? pairs * a.nbf * 4 : 0));
    return at;
}

// mode: 0 f32, 1 one-word, 2 two-word.  route: the router's logits, choices and
// gates; experts: the projections (with the router's choices, or given ones).
hipError_t launch_moe(int mode, const MoeArgs &a, bool route, bool experts, hipStream_t stream);

}  // namespace q8
