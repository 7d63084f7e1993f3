// moe_abi.cpp -- the C ABI of the mixture-of-experts layer (q8_decode.h):
// argument validation, then 64-row slices on the caller's stream.  As in
// abi.cpp, nothing here allocates, synchronizes or reads device memory, and
// errors are returned by name before anything is enqueued.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/q8_decode.h"
#include "moe.h"
#include "ranges.h"

namespace {

constexpr int64_t kMaxDim = 65536;                    // k and ff
constexpr int64_t kMaxLayerBlocks = int64_t(1) << 31;  // blocks of one of the three matrices (73 GB)
constexpr int64_t kMaxRows = int64_t(1) << 20;

q8_status check_layer(const q8_moe_layer *l, int64_t rows) {
    if (!l) return Q8_E_NULL;
    if (l->mode != Q8_ACT_F32 && l->mode != Q8_ACT_I8 && l->mode != Q8_ACT_I8X2) return Q8_E_MODE;
    if (rows < 0 || rows > kMaxRows) return Q8_E_SHAPE;
    if (l->n_experts < 1 || l->n_experts > q8::kMoeMaxExperts) return Q8_E_SHAPE;
    if (l->top_k < 1 || l->top_k > std::min(l->n_experts, q8::kMoeMaxTopK)) return Q8_E_SHAPE;
    for (int64_t d : {l->k, l->ff})
        if (d < 64 || d % 64 != 0 || d > kMaxDim) return Q8_E_SHAPE;
    if (l->n_experts > kMaxLayerBlocks / (l->ff * (l->k / 32))) return Q8_E_SHAPE;
    return Q8_OK;
}

// The layer's sizes for a slice of `rows` rows.
q8::MoeArgs sizes_of(const q8_moe_layer *l, int rows) {
    q8::MoeArgs a = {};
    a.rows = rows;
    a.experts = l->n_experts;
    a.top_k = l->top_k;
    a.renormalize = l->renormalize != 0;
    a.k = static_cast<int>(l->k);
    a.nbk = static_cast<int>(l->k / 32);
    a.ff = static_cast<int>(l->ff);
    a.nbf = static_cast<int>(l->ff / 32);
    return a;
}

// The three entry points: route and/or experts over 64-row slices.
q8_status moe(const q8_moe_layer *l, const float *x, int64_t rows, const float *residual, float *y, int32_t *ids,
              float *gates, void *workspace, int64_t workspace_bytes, void *stream, bool route, bool experts) {
    if (q8_status s = check_layer(l, rows); s != Q8_OK) return s;
    if (!x || !ids || !gates || !workspace) return Q8_E_NULL;
    if (route && !l->router) return Q8_E_NULL;
    if (experts && (!l->w_gate || !l->w_up || !l->w_down || !y)) return Q8_E_NULL;
    if (!q8::aligned_to(x, 16) || !q8::aligned_to(ids, 4) || !q8::aligned_to(gates, 4) || !q8::aligned_to(workspace, 16)) return Q8_E_ALIGN;
    if (route && !q8::aligned_to(l->router, 16)) return Q8_E_ALIGN;
    if (experts && (!q8::aligned_to(l->w_gate, 4) || !q8::aligned_to(l->w_up, 4) || !q8::aligned_to(l->w_down, 4) || !q8::aligned_to(y, 4) ||
                    !q8::aligned_to(residual, 4)))
        return Q8_E_ALIGN;
    const int64_t need = q8_moe_workspace_bytes(l, rows);
    if (workspace_bytes < need) return Q8_E_SHAPE;
    const int64_t wbytes = int64_t(l->n_experts) * l->ff * (l->k / 32) * 34;
    const q8::Range rx{x, rows * l->k * 4}, ry{experts ? y : nullptr, rows * l->k * 4},
        rres{experts ? residual : nullptr, rows * l->k * 4}, rids{ids, rows * l->top_k * 4},
        rgates{gates, rows * l->top_k * 4}, rws{workspace, need},
        rr{route ? l->router : nullptr, int64_t(l->n_experts) * l->k * 4},
        rg{experts ? l->w_gate : nullptr, wbytes}, ru{experts ? l->w_up : nullptr, wbytes},
        rd{experts ? l->w_down : nullptr, wbytes};
    const q8::Range inputs[] = {rx, rr, rg, ru, rd};
    for (const q8::Range &in : inputs)
        if (q8::overlaps(ry, in) || q8::overlaps(rws, in) || (route && (q8::overlaps(rids, in) || q8::overlaps(rgates, in))))
            return Q8_E_ALIAS;
    if (q8::overlaps(ry, rids) || q8::overlaps(ry, rgates) || q8::overlaps(rws, ry) || q8::overlaps(rws, rres) || q8::overlaps(rws, rids) ||
        q8::overlaps(rws, rgates))
        return Q8_E_ALIAS;
    if (route && (q8::overlaps(rids, rgates) || q8::overlaps(rids, rres) || q8::overlaps(rgates, rres))) return Q8_E_ALIAS;
    if (residual != y && q8::overlaps(ry, rres)) return Q8_E_ALIAS;
    for (int64_t r0 = 0; r0 < rows; r0 += q8::kMoeSlice) {
        q8::MoeArgs a = sizes_of(l, static_cast<int>(std::min<int64_t>(q8::kMoeSlice, rows - r0)));
        q8::moe_layout(a, static_cast<uint8_t *>(workspace), l->mode);
        a.x = x + r0 * l->k;
        a.router = l->router;
        a.w_gate = static_cast<const uint8_t *>(l->w_gate);
        a.w_up = static_cast<const uint8_t *>(l->w_up);
        a.w_down = static_cast<const uint8_t *>(l->w_down);
        a.residual = residual ? residual + r0 * l->k : nullptr;
        a.y = y ? y + r0 * l->k : nullptr;
        a.ids = ids + r0 * l->top_k;
        a.gates = gates + r0 * l->top_k;
        if (q8::launch_moe(l->mode, a, route, experts, reinterpret_cast<hipStream_t>(stream)) != hipSuccess)
            return Q8_E_HIP;
    }
    return Q8_OK;
}

}  // namespace

extern "C" {

int64_t q8_moe_workspace_bytes(const q8_moe_layer *layer, int64_t rows) {
    if (check_layer(layer, rows) != Q8_OK) return 0;
    q8::MoeArgs a = sizes_of(layer, static_cast<int>(std::min<int64_t>(q8::kMoeSlice, rows)));
    return q8::moe_layout(a, nullptr, layer->mode);
}

q8_status q8_moe_route(const q8_moe_layer *layer, const float *x, int64_t rows, int32_t *ids, float *gates,
                       void *workspace, int64_t workspace_bytes, void *stream) {
    return moe(layer, x, rows, nullptr, nullptr, ids, gates, workspace, workspace_bytes, stream, true, false);
}

q8_status q8_moe_experts(const q8_moe_layer *layer, const float *x, int64_t rows, const int32_t *ids,
                         const float *gates, const float *residual, float *y, void *workspace,
                         int64_t workspace_bytes, void *stream) {
    // the choices are read only: the router, which would write them, does not run
    return moe(layer, x, rows, residual, y, const_cast<int32_t *>(ids), const_cast<float *>(gates), workspace,
               workspace_bytes, stream, false, true);
}

q8_status q8_moe(const q8_moe_layer *layer, const float *x, int64_t rows, const float *residual, float *y,
                 int32_t *ids, float *gates, void *workspace, int64_t workspace_bytes, void *stream) {
    return moe(layer, x, rows, residual, y, ids, gates, workspace, workspace_bytes, stream, true, true);
}

}  // extern "C"
