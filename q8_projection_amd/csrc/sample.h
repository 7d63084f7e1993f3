// sample.h -- arguments of the sampler's kernels and their workspace.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q8 {

constexpr int64_t kSampleMaxN = (int64_t(1) << 19) - 1;  // sums of n weights of at most 2^44 fit 63 bits
constexpr int64_t kSampleMaxRows = int64_t(1) << 16;
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
    float *submax;             // workspace [rows][nsub]
    int nsub;
};

// Places the workspace's parts (base may be null: sizes only); returns its bytes.
inline int64_t sample_layout(SampleArgs &a, uint8_t *base) {
    a.nsub = (a.n + kSubBlock - 1) / kSubBlock;
    a.submax = reinterpret_cast<float *>(base);
    return (static_cast<int64_t>(a.rows) * a.nsub * 4 + 255) / 256 * 256;
}

hipError_t launch_sample(const SampleArgs &a, hipStream_t stream);

}  // namespace q8
