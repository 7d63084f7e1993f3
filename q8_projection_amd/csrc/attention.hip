// attention.hip -- attention of f32 queries over the quantized cache (q8_cache.h).
//
// One wave a row and query head, one tile of 32 tokens at a time with the running
// maximum and sum of the softmax: a lane's token for the scores, a lane's dimensions for
// the values.
#include <algorithm>

#include "cache.h"
#include "device.h"

namespace q8 {
namespace {

constexpr int kWaves = 4;

template <int BITS, int D>
__global__ __launch_bounds__(64 * kWaves) void attention_kernel(AttentionArgs a) {
    using T = Tile<BITS, D>;
    __shared__ float qs[kWaves][D];
    __shared__ float ps[kWaves][kTileTokens];
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int64_t wave = wid + int64_t(blockIdx.x) * kWaves;
    const int64_t rest = wave / a.heads;
    const int h = static_cast<int>(wave - rest * a.heads);
    const int s = static_cast<int>(rest / a.c.max_rows), i = static_cast<int>(rest % a.c.max_rows);
    if (s >= a.c.sequences) return;
    const Rows rows = sequence_rows(a.c, s);
    if (i >= rows.n) return;
    const int64_t row = rows.first + i;
    const int at = rows.at + i;  // the row's token
    float *q = qs[wid], *p = ps[wid];
    for (int j = lane; j < D; j += 64) q[j] = a.q[row * a.q_ld + int64_t(h) * D + j] * a.scale;
    wave_lds_sync();
    const int end = min(at + 1, rows.end), begin = a.window ? max(at - a.window + 1, 0) : 0;
    const int tok = lane & 31, half = lane >> 5;
    float top = -3e38f, total = 0.0f, acc[D / 64] = {};
    for (int t = begin / kTileTokens; t * kTileTokens < end; ++t) {
        const uint8_t *tile = tile_at<BITS, D>(a.c, s, t, h / a.group);
        if (!tile) continue;
        float z = 0.0f;
        for (int blk = half * (D / 64); blk < (half + 1) * (D / 64); ++blk) {
            const uint32_t word = reinterpret_cast<const uint16_t *>(tile + T::kKeyWords)[key_word(tok, blk, T::kBlocks)];
            for (int e = 0; e < 32; ++e) {
                const int d = blk * 32 + e;
                const uint32_t byte = tile[tok * T::kRow + d * BITS / 8];
                z += q[d] * value_of<BITS>(word, BITS == 8 ? byte : byte >> (4 * (d & 1)) & 15u);
            }
        }
        z += __shfl_xor(z, 32, 64);
        const int token = t * kTileTokens + tok;
        z = token >= begin && token < end ? z : -INFINITY;
        const float most = fmaxf(top, wave_max(z));
        const float e = expf(z - most), keep = expf(top - most);
        top = most;
        total *= keep;
        for (int u = 0; u < D / 64; ++u) acc[u] *= keep;
        if (half == 0) p[tok] = e;
        wave_lds_sync();
        for (int n = 0; n < kTileTokens; ++n) {
            if (p[n] == 0.0f) continue;  // a masked token's codes may be anything
            total += p[n];
            for (int u = 0; u < D / 64; ++u) {
                const int d = u * 64 + lane, g = n >> 3, b = n & 3, w = n >> 2 & 1;
                const uint32_t word = reinterpret_cast<const uint16_t *>(tile + T::kValueWords)[value_word(n, d / 32)];
                const int place = BITS == 4 ? (((d / 64 * 4 + g) * 16 + d % 16) * 4 + d / 16 % 4) * 4 + (n & 7) / 2
                                            : (((d / 32 * 4 + g) * 16 + d % 16) * 2 + d / 16 % 2) * 8 + b * 2 + w;
                const uint32_t byte = tile[T::kValues + place];
                acc[u] += p[n] * value_of<BITS>(word, BITS == 8 ? byte : byte >> (4 * (n & 1)) & 15u);
            }
        }
        wave_lds_sync();
    }
    for (int u = 0; u < D / 64; ++u)
        a.out[(row * a.heads + h) * D + u * 64 + lane] = total > 0 ? acc[u] / total : 0.0f;
    if (a.lse && lane == 0) a.lse[row * a.heads + h] = total > 0 ? top + logf(total) : -INFINITY;
}

template <int BITS, int D>
hipError_t launch(const AttentionArgs &a, hipStream_t stream) {
    const int64_t waves = int64_t(a.c.sequences) * a.c.max_rows * a.heads;
    attention_kernel<BITS, D><<<dim3(static_cast<uint32_t>((waves + kWaves - 1) / kWaves)), dim3(64 * kWaves), 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

int64_t attention_workspace(int dim, const AttentionArgs &a) {
    AttentionArgs b = a;
    b.c.max_rows = std::min(b.c.max_rows, std::max(kFewRows / b.group, 1));
    return few_workspace(dim, b);
}

hipError_t launch_attention(int bits, int dim, const AttentionArgs &a, void *workspace, hipStream_t stream) {
    if (int64_t(a.c.max_rows) * a.group <= kFewRows) return launch_few(bits, dim, a, workspace, stream);
    if (bits == 4)
        return dim == 64 ? launch<4, 64>(a, stream) : dim == 128 ? launch<4, 128>(a, stream) : launch<4, 256>(a, stream);
    return dim == 64 ? launch<8, 64>(a, stream) : dim == 128 ? launch<8, 128>(a, stream) : launch<8, 256>(a, stream);
}

}  // namespace q8
