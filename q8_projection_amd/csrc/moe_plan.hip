// moe_plan.hip -- the first steps of the mixture-of-experts layer: the router's
// logits, the activation quantization of x, the choice of experts and the plan
// that groups the chosen (token, expert) pairs by expert.
#include "actquant.h"
#include "device.h"
#include "moe.h"
#include "moe_kernels.h"

#pragma clang fp contract(off)

namespace q8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTokenGroup = 8;  // tokens one workgroup dots a router row with

// z[t][e] for one expert and up to 8 tokens, by one workgroup: threads stride over k
// four values at a time (every product exact in f64, 24 x 24 bits, and every sum in
// f64), the waves' sums are added in wave order.
__device__ __forceinline__ void route_logits(const MoeArgs &a, int e, int t0) {
    __shared__ double part[kWaves][kTokenGroup];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const float4 *r = reinterpret_cast<const float4 *>(a.router + static_cast<int64_t>(e) * a.k);
    const int n4 = a.k / 4;
    const int nt = min(kTokenGroup, a.rows - t0);
    const float4 *x = reinterpret_cast<const float4 *>(a.x + static_cast<int64_t>(t0) * a.k);
    double acc[kTokenGroup];
#pragma unroll
    for (int t = 0; t < kTokenGroup; ++t) acc[t] = 0.0;
#pragma unroll 2
    for (int i = threadIdx.x; i < n4; i += kThreads) {
        const float4 w = r[i];
#pragma unroll
        for (int t = 0; t < kTokenGroup; ++t) {
            if (t >= nt) break;
            const float4 v = x[static_cast<int64_t>(t) * n4 + i];
            acc[t] = __builtin_fma(static_cast<double>(w.x), static_cast<double>(v.x), acc[t]);
            acc[t] = __builtin_fma(static_cast<double>(w.y), static_cast<double>(v.y), acc[t]);
            acc[t] = __builtin_fma(static_cast<double>(w.z), static_cast<double>(v.z), acc[t]);
            acc[t] = __builtin_fma(static_cast<double>(w.w), static_cast<double>(v.w), acc[t]);
        }
    }
#pragma unroll
    for (int t = 0; t < kTokenGroup; ++t) {
        if (t >= nt) break;
        const double z = wave_sum(acc[t]);
        if (lane == 0) part[wave][t] = z;
    }
    __syncthreads();
    const int t = threadIdx.x;
    if (t < nt) {
        const double z = (part[0][t] + part[1][t]) + (part[2][t] + part[3][t]);
        a.logits[static_cast<int64_t>(t0 + t) * a.experts + e] = static_cast<float>(z);
    }
}

// Workgroups [0, quant_wgs) quantize x, the rest take router rows.
template <int WORDS>
__global__ __launch_bounds__(kThreads) void moe_prepare_kernel(MoeArgs a, int quant_wgs) {
    if constexpr (WORDS > 0) {
        if (static_cast<int>(blockIdx.x) < quant_wgs) {
            const int t = static_cast<int>(blockIdx.x) * kThreads + threadIdx.x;
            const int blk = t / kQuantLanes, part = t % kQuantLanes;
            const bool valid = blk < a.rows * a.nbk;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (valid) v = reinterpret_cast<const float4 *>(a.x)[t];
            uint32_t h4, l4;
            const float s = quantize4<WORDS>(v, h4, l4);
            if (!valid) return;
            uint32_t *rec = reinterpret_cast<uint32_t *>(a.xq + static_cast<int64_t>(blk) * (WORDS * 32));
            rec[part] = h4;
            if (WORDS == 2) rec[8 + part] = l4;
            if (part == 0) a.xs[blk] = s;
            return;
        }
    }
    const int item = static_cast<int>(blockIdx.x) - quant_wgs;
    route_logits(a, item % a.experts, item / a.experts * kTokenGroup);
}

// The top_k largest logits of a token, in descending order, the lowest expert
// among equals; one wave, experts dealt to lanes e = lane + 64 j.  A token whose
// logits run out (NaN) gets id -1 and gate 0.
__device__ __forceinline__ void choose(const MoeArgs &a, int t, int lane) {
    constexpr int J = kMoeMaxExperts / 64;
    const float *z = a.logits + static_cast<int64_t>(t) * a.experts;
    float v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = lane + 64 * j;
        v[j] = e < a.experts ? z[e] : -__builtin_inff();
    }
    float top = 0.f;
    double sum = 0.0;       // of the exps of the chosen, in order
    float mine = 0.f;       // lane i keeps choice i
    int mine_id = -1;
    uint32_t taken = 0;     // this lane's chosen j
    const int nj = (a.experts + 63) / 64;
    for (int i = 0; i < a.top_k; ++i) {
        float bv = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (j >= nj) break;
            if (!((taken >> j) & 1)) bv = fmaxf(bv, v[j]);
        }
        bv = wave_max(bv);
        // the lowest expert that has it
        int be = -1;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            if (j >= nj || be >= 0) break;
            const uint64_t has = __ballot(lane + 64 * j < a.experts && !((taken >> j) & 1) && v[j] == bv);
            if (has) be = 64 * j + __builtin_ctzll(has);
        }
        if (be < 0) break;
        if ((be & 63) == lane) taken |= 1u << (be >> 6);
        if (i == 0) top = bv;
        sum += exp(static_cast<double>(bv) - static_cast<double>(top));
        if (lane == i) {
            mine = bv;
            mine_id = be;
        }
    }
    if (!a.renormalize) {
        double s = 0.0;
#pragma unroll
        for (int j = 0; j < J; ++j)
            if (lane + 64 * j < a.experts) s += exp(static_cast<double>(v[j]) - static_cast<double>(top));
        sum = wave_sum(s);
    }
    if (lane < a.top_k) {
        const double p = mine_id < 0 ? 0.0 : exp(static_cast<double>(mine) - static_cast<double>(top)) / sum;
        a.ids[static_cast<int64_t>(t) * a.top_k + lane] = mine_id;
        a.gates[static_cast<int64_t>(t) * a.top_k + lane] = static_cast<float>(p);
    }
}

constexpr int kPlanThreads = 1024;

// One workgroup: the choices (route), then the plan (experts): per expert the
// set of its tokens as a bit mask (or-ed, so the order of the threads does not
// matter), the active experts in ascending order, and each pair's token and
// gate at a place its mask gives.
__global__ __launch_bounds__(kPlanThreads) void moe_plan_kernel(MoeArgs a, int route, int plan) {
    __shared__ unsigned long long mask[kMoeMaxExperts];
    __shared__ uint32_t scan[kMoeMaxExperts];
    const int tid = threadIdx.x;
    if (route) {
        for (int t = tid >> 6; t < a.rows; t += kPlanThreads / 64) choose(a, t, tid & 63);
        __threadfence_block();
    }
    if (!plan) return;
    if (tid < kMoeMaxExperts) mask[tid] = 0;
    __syncthreads();
    const int pairs = a.rows * a.top_k;
    const int t = tid / a.top_k;
    int id = -1;
    if (tid < pairs) {
        id = a.ids[tid];
        if (id < 0 || id >= a.experts) id = -1;
        if (id >= 0) atomicOr(&mask[id], 1ull << t);
    }
    __syncthreads();
    // inclusive scan of (active experts << 16 | pairs)
    uint32_t own = 0;
    if (tid < kMoeMaxExperts) {
        const int c = __popcll(mask[tid]);
        own = (c > 0 ? 1u << 16 : 0u) + static_cast<uint32_t>(c);
        scan[tid] = own;
    }
    for (int off = 1; off < kMoeMaxExperts; off <<= 1) {
        __syncthreads();
        const uint32_t add = tid < kMoeMaxExperts && tid >= off ? scan[tid - off] : 0u;
        __syncthreads();
        if (tid < kMoeMaxExperts) scan[tid] += add;
    }
    __syncthreads();
    if (tid < kMoeMaxExperts && own) {
        const uint32_t before = scan[tid] - own;
        MoeEntry &en = a.plan->entry[before >> 16];
        en.expert = tid;
        en.offset = static_cast<int32_t>(before & 0xffffu);
        en.mask = mask[tid];
    }
    if (tid == 0) a.plan->n_active = static_cast<int32_t>(scan[kMoeMaxExperts - 1] >> 16);
    if (id >= 0) {
        // a repeated choice counts once, with the sum of its gates in slot order
        bool first = true;
        double gate = 0.0;
        for (int s = 0; s < a.top_k; ++s) {
            const int p = t * a.top_k + s;
            if (a.ids[p] != id) continue;
            if (p < tid) first = false;
            gate += static_cast<double>(a.gates[p]);
        }
        if (first) {
            const int c = __popcll(mask[id]);
            const int at = static_cast<int>((scan[id] & 0xffffu)) - c + __popcll(mask[id] & ((1ull << t) - 1));
            a.plan->pair_token[at] = t;
            a.plan->pair_gate[at] = gate;
        }
    }
}

}  // namespace

hipError_t launch_moe(int mode, const MoeArgs &a, bool route, bool experts, hipStream_t stream) {
    const int quant_wgs =
        experts && mode != 0 ? (a.rows * a.nbk * kQuantLanes + kThreads - 1) / kThreads : 0;
    const int groups = (a.rows + kTokenGroup - 1) / kTokenGroup;
    const int route_wgs = route ? a.experts * groups : 0;
    if (quant_wgs + route_wgs > 0) {
        const dim3 grid(quant_wgs + route_wgs);
        if (mode == 2)
            moe_prepare_kernel<2><<<grid, kThreads, 0, stream>>>(a, quant_wgs);
        else if (mode == 1)
            moe_prepare_kernel<1><<<grid, kThreads, 0, stream>>>(a, quant_wgs);
        else
            moe_prepare_kernel<0><<<grid, kThreads, 0, stream>>>(a, quant_wgs);
        if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    }
    moe_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, route, experts);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || !experts) return e;
    return launch_moe_experts(mode, a, stream);
}

}  // namespace q8
