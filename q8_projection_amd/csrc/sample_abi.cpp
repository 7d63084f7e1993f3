// sample_abi.cpp -- the C ABI of the sampler (q8_decode.h): argument validation,
// then the launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/q8_decode.h"
#include "ranges.h"
#include "sample.h"

extern "C" {

int64_t q8_sample_workspace_bytes(int64_t rows, int64_t n) {
    if (rows < 0 || rows > q8::kSampleMaxRows || n < 1 || n > q8::kSampleMaxN) return 0;
    q8::SampleArgs a = {};
    a.rows = static_cast<int>(std::min<int64_t>(rows, q8::kSampleSlice));
    a.n = static_cast<int>(n);
    return q8::sample_layout(a, nullptr);
}

q8_status q8_sample(const float *logits, int64_t ld, int64_t rows, int64_t n, const float *temperature,
                    const int32_t *top_k, const float *top_p, const float *min_p, const float *u, int32_t *idx,
                    float *prob, void *workspace, int64_t workspace_bytes, void *stream) {
    if (rows < 0 || rows > q8::kSampleMaxRows || n < 1 || n > q8::kSampleMaxN) return Q8_E_SHAPE;
    if (ld < n || ld > (int64_t(1) << 40)) return Q8_E_SHAPE;
    if (!logits || !u || !idx || !workspace) return Q8_E_NULL;
    for (const void *p : {static_cast<const void *>(logits), static_cast<const void *>(temperature),
                          static_cast<const void *>(top_k), static_cast<const void *>(top_p),
                          static_cast<const void *>(min_p), static_cast<const void *>(u),
                          static_cast<const void *>(idx), static_cast<const void *>(prob)})
        if (!q8::aligned_to(p, 4)) return Q8_E_ALIGN;
    if (!q8::aligned_to(workspace, 16)) return Q8_E_ALIGN;
    const int64_t need = q8_sample_workspace_bytes(rows, n);
    if (workspace_bytes < need) return Q8_E_SHAPE;
    const int64_t bytes = rows * 4;
    const q8::Range outs[] = {{idx, bytes}, {prob, bytes}, {workspace, need}};
    const q8::Range ins[] = {{logits, rows ? ((rows - 1) * ld + n) * 4 : 0},
                             {temperature, bytes}, {top_k, bytes}, {top_p, bytes}, {min_p, bytes}, {u, bytes}};
    for (int i = 0; i < 3; ++i) {
        for (const q8::Range &in : ins)
            if (q8::overlaps(outs[i], in)) return Q8_E_ALIAS;
        for (int j = 0; j < i; ++j)
            if (q8::overlaps(outs[i], outs[j])) return Q8_E_ALIAS;
    }
    if (rows == 0) return Q8_OK;
    for (int64_t r0 = 0; r0 < rows; r0 += q8::kSampleSlice) {
        q8::SampleArgs a = {};
        a.logits = logits + r0 * ld;
        a.ld = ld;
        a.n = static_cast<int>(n);
        a.rows = static_cast<int>(std::min<int64_t>(rows - r0, q8::kSampleSlice));
        a.temperature = temperature ? temperature + r0 : nullptr;
        a.top_k = top_k ? top_k + r0 : nullptr;
        a.top_p = top_p ? top_p + r0 : nullptr;
        a.min_p = min_p ? min_p + r0 : nullptr;
        a.u = u + r0;
        a.idx = idx + r0;
        a.prob = prob ? prob + r0 : nullptr;
        q8::sample_layout(a, static_cast<uint8_t *>(workspace));
        if (q8::launch_sample(a, reinterpret_cast<hipStream_t>(stream)) != hipSuccess) return Q8_E_HIP;
    }
    return Q8_OK;
}

}  // extern "C"
