// sample.h -- arguments of the sampler's kernels and their workspace.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace q8 {

constexpr int64_t kSampleMaxN = (int64_t(1) << 19) - 1;  // sums of n weights of at most 2^44 fit 63 bits
constexpr int64_t kSampleMaxRows = int64_t(1) << 16;
constexpr int kSampleSlice = 1024;  // rows of one pass (a histogram each in the workspace)
constexpr int kSubBlock = 64;                            // logits per stored maximum

struct SampleArgs {
    const float *logits;       // [rows], row stride ld
    int64_t ld;
    int n;
    int rows;
    const float *temperature;  // [rows]
    const int32_t *top_k;      // [rows] or null: all
    const float *top_p;        // [rows] or null: 1
    const float *min_p;        // [rows] or null: 0
    const float *u;            // [rows]
    int32_t *idx;              // [rows]
    float *prob;               // [rows] or null
    int nsub;                  // maxima a row
    int segments;              // workgroups that share a row's histogram
    // workspace
    struct RowState *state;    // [rows]
    unsigned long long *sums;  // [rows][segments][kSampleSums]: the segments' histograms
    unsigned long long *near;  // [rows][kNear]: gathered tokens
    int gathers;               // workgroups that gather a row's tokens, a power of two
    float *submax;             // [rows][nsub]
    float *wavemax;            // [rows][nwave]: maxima of 1024 logits
    int nwave;
    int segment;               // logits of one segment
};

// How far a row is (cleared by the first kernel of a call).
struct RowState {
    uint32_t phase;    // 0: every segment has its histogram; 1: drawn; 2: segment 0 has the whole row's
    uint32_t fill;     // tokens gathered
    uint32_t arrived;  // workgroups that have gathered
    uint32_t pad;
};

constexpr int kNear = 1024;
constexpr int kSampleBins = 2048;
// a histogram: weight sums of the bins, counts of the bins (32 bits each),
// and the sum of the weights that min-p keeps
constexpr int kSampleSums = kSampleBins + kSampleBins / 2 + 1;
constexpr int kSegment = 4096;  // logits one workgroup adds up, at least
constexpr int kHistogramWgs = 256;  // workgroups that make histograms: one a CU
// Workgroups that gather a call's rows, and logits one takes alone (64 mixed rows of 151936:
// 29 us; with up to 512 workgroups 43, with 128 36)
constexpr int kGatherWgs = 256, kGatherLogits = 65536;
constexpr int kMaxWgLogits = 4096;  // logits of one workgroup of the maxima's kernel, 1024 a wave

// Places the workspace's parts (base may be null: sizes only); returns its bytes.
inline int64_t sample_layout(SampleArgs &a, uint8_t *base) {
    a.nsub = (a.n + kSubBlock - 1) / kSubBlock;
    // Enough segments for a workgroup a CU (more do not fit), no more: each costs the row's
    // maximum, an empty histogram and the reading of its own by the last kernel.
    const int most = std::min(16, (a.n + kSegment - 1) / kSegment);
    const int want = a.rows > 0 ? (kHistogramWgs + a.rows - 1) / a.rows : 1;
    a.segments = std::min(want, most);
    a.segment = ((a.n + a.segments - 1) / a.segments + kSegment - 1) / kSegment * kSegment;
    a.segments = (a.n + a.segment - 1) / a.segment;
    a.nwave = (a.n + kMaxWgLogits - 1) / kMaxWgLogits * 4;
    int64_t at = 0;
    auto take = [&](int64_t bytes) {
        uint8_t *p = base ? base + at : nullptr;
        at += (bytes + 255) / 256 * 256;
        return p;
    };
    a.gathers = 1;
    while (a.gathers < 8 && 2 * a.gathers * a.rows <= kGatherWgs && a.n / a.gathers > kGatherLogits) a.gathers *= 2;
    // Room for what any smaller call needs as well: the sizes grow with rows and n.
    const int64_t histograms = std::min(int64_t(a.rows) * most, int64_t(a.rows) + kHistogramWgs);
    const int64_t lists = a.n > kGatherLogits ? std::min(a.rows, kGatherWgs / 2) : 0;
    a.state = reinterpret_cast<RowState *>(take(sizeof(RowState) * int64_t(a.rows)));
    a.sums = reinterpret_cast<unsigned long long *>(take(8 * kSampleSums * histograms));
    a.near = reinterpret_cast<unsigned long long *>(take(8 * kNear * lists));
    a.submax = reinterpret_cast<float *>(take(int64_t(4) * a.rows * a.nsub));
    a.wavemax = reinterpret_cast<float *>(take(int64_t(4) * a.rows * a.nwave));
    return at;
}

hipError_t launch_sample(const SampleArgs &a, hipStream_t stream);

}  // namespace q8
