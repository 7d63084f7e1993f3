// moe_plan.hip -- the first launch of the mixture-of-experts layer: the router's
// logits, the activation quantization of x, the choice of experts and the plan
// that groups the chosen (token, expert) pairs by expert.
//
// One launch for the four: the last workgroup of a group of tokens to finish its
// logits makes their choices, the last of those the plan.  Launches of their own would
// each add a start to a layer that takes 15 us at its smallest.  The logits are f64 sums rounded to f32 once, so
// that the choice can be checked from them; gates are f64 quotients rounded once.
// What bounds it is the chain of these steps, not the router's bytes: one token of 64
// experts 6.8 us, 64 tokens 15 us (k 2048), given choices 3.8 us.
#include "actquant.h"
#include "device.h"
#include "moe.h"
#include "moe_kernels.h"

#pragma clang fp contract(off)

namespace q8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTokenGroup = 4;  // tokens one workgroup dots a router row with, and then a wave each chooses for
static_assert((kMoeSlice / kTokenGroup + 1) * kMoeCounterStride <= kMoeTileCounter,
              "a counter for each token group and one more, before the tiles' counters");

// z[t][e] for one expert and up to 4 tokens, by one workgroup: threads stride over k
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
        __hip_atomic_store(a.logits + static_cast<int64_t>(t0 + t) * a.experts + e, static_cast<float>(z),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// The top_k largest logits of a token, in descending order, the lowest expert
// among equals; one wave, experts dealt to lanes e = lane + 64 j.  A token whose
// logits run out (NaN) gets id -1 and gate 0.  Lane i returns choice i.
template <int J>
__device__ __forceinline__ void choose(const MoeArgs &a, int t, int lane, int &id, float &gate) {
    const float *z = a.logits + static_cast<int64_t>(t) * a.experts;
    float v[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int e = lane + 64 * j;
        v[j] = __hip_atomic_load(z + min(e, a.experts - 1), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    uint32_t open = 0;  // this lane's j that are not chosen yet
#pragma unroll
    for (int j = 0; j < J; ++j) open |= lane + 64 * j < a.experts ? 1u << j : 0u;
    const uint32_t all = open;
    float mine = 0.f;
    id = -1;
    for (int i = 0; i < a.top_k; ++i) {
        float bv = -__builtin_inff();
#pragma unroll
        for (int j = 0; j < J; ++j) bv = fmaxf(bv, (open >> j) & 1 ? v[j] : -__builtin_inff());
        bv = wave_max(bv);
        int be = -1;  // the lowest expert that has it
#pragma unroll
        for (int j = J - 1; j >= 0; --j) {
            const uint64_t has = __ballot(((open >> j) & 1) && v[j] == bv);
            if (has) be = 64 * j + __builtin_ctzll(has);
        }
        if (be < 0) break;
        if ((be & 63) == lane) open &= ~(1u << (be >> 6));
        if (lane == i) {
            mine = bv;
            id = be;
        }
    }
    const double top = static_cast<double>(__builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, mine), 0)));
    const double mine_exp = id < 0 ? 0.0 : exp(static_cast<double>(mine) - top);
    double sum = 0.0;
    if (a.renormalize) {
        for (int i = 0; i < a.top_k; ++i) sum += readlane_f64(mine_exp, i);
    } else {
#pragma unroll
        for (int j = 0; j < J; ++j)
            if ((all >> j) & 1) sum += exp(static_cast<double>(v[j]) - top);
        sum = wave_sum(sum);
    }
    gate = static_cast<float>(id < 0 ? 0.0 : mine_exp / sum);
}

__device__ __forceinline__ void choose(const MoeArgs &a, int t, int lane, int &id, float &gate) {
    if (a.experts <= 64)
        choose<1>(a, t, lane, id, gate);
    else if (a.experts <= 128)
        choose<2>(a, t, lane, id, gate);
    else
        choose<kMoeMaxExperts / 64>(a, t, lane, id, gate);
}

// The plan of a single token from its choices (all different, lane i has choice i):
// its experts in ascending order.
__device__ __forceinline__ void plan_one(const MoeArgs &a, int lane, int id, float gate) {
    int before = 0, n = 0;
    for (int i = 0; i < a.top_k; ++i) {
        const int other = __builtin_amdgcn_readlane(id, i);
        n += other >= 0;
        before += other >= 0 && other < id;
    }
    if (lane < a.top_k && id >= 0) {
        MoeEntry &en = a.plan->entry[before];
        en.expert = id;
        en.offset = before;
        en.mask = 1;
        a.plan->pair_token[before] = 0;
        a.plan->pair_gate[before] = static_cast<double>(gate);
    }
    if (lane == 0) a.plan->n_active = n;
}

// The plan, by one workgroup: per expert the set of its tokens as a bit mask (or-ed,
// so the order of the threads does not matter), the active experts in ascending
// order, and each pair's token and gate at a place that its mask gives.
__device__ __forceinline__ void make_plan(const MoeArgs &a) {
    __shared__ unsigned long long mask[kMoeMaxExperts];
    __shared__ uint32_t before[kMoeMaxExperts];  // (active experts << 16 | pairs) before this one
    __shared__ uint32_t wave_total[kWaves];
    __shared__ int32_t ids[kMoeMaxPairs];
    __shared__ float gates[kMoeMaxPairs];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int pairs = a.rows * a.top_k;
    constexpr int kPer = kMoeMaxPairs / kThreads;
    int32_t id[kPer];
    float gate[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {  // every load in flight at once
        const int p = min(tid + i * kThreads, pairs - 1);
        id[i] = __hip_atomic_load(a.ids + p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        gate[i] = __hip_atomic_load(a.gates + p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    for (int e = tid; e < a.experts; e += kThreads) mask[e] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int p = tid + i * kThreads;
        if (p >= pairs) break;
        const bool ok = id[i] >= 0 && id[i] < a.experts;
        ids[p] = ok ? id[i] : -1;
        gates[p] = gate[i];
        if (ok) atomicOr(&mask[id[i]], 1ull << (p / a.top_k));
    }
    __syncthreads();
    // each thread has consecutive experts; their totals are scanned over the workgroup
    const int per = (a.experts + kThreads - 1) / kThreads;
    uint32_t own = 0;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        const int c = e < a.experts ? __popcll(mask[e]) : 0;
        own += (c > 0 ? 1u << 16 : 0u) + static_cast<uint32_t>(c);
    }
    uint32_t run = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t o = __shfl_up(run, off, 64);
        if (lane >= off) run += o;
    }
    if (lane == 63) wave_total[wave] = run;
    __syncthreads();
    for (int w = 0; w < wave; ++w) run += wave_total[w];
    if (tid == kThreads - 1) a.plan->n_active = static_cast<int32_t>(run >> 16);
    run -= own;
    for (int i = 0; i < per; ++i) {
        const int e = tid * per + i;
        const int c = e < a.experts ? __popcll(mask[e]) : 0;
        if (c > 0) {
            before[e] = run;
            MoeEntry &en = a.plan->entry[run >> 16];
            en.expert = e;
            en.offset = static_cast<int32_t>(run & 0xffffu);
            en.mask = mask[e];
            run += (1u << 16) + static_cast<uint32_t>(c);
        }
    }
    __syncthreads();
    for (int p = tid; p < pairs; p += kThreads) {
        const int e = ids[p];
        if (e < 0) continue;
        // a repeated choice counts once, with the sum of its gates in slot order
        const int t = p / a.top_k;
        bool first = true;
        double sum = 0.0;
        for (int q = t * a.top_k; q < (t + 1) * a.top_k; ++q) {
            if (ids[q] != e) continue;
            if (q < p) first = false;
            sum += static_cast<double>(gates[q]);
        }
        if (first) {
            const int at = static_cast<int>(before[e] & 0xffffu) + __popcll(mask[e] & ((1ull << t) - 1));
            a.plan->pair_token[at] = t;
            a.plan->pair_gate[at] = sum;
        }
    }
}

// Counts this workgroup in; true for the one that makes `total`, which puts the counter
// back to zero.  What the workgroup has stored at agent scope is complete by then (the
// waits), and the last one reads it at agent scope.
__device__ __forceinline__ bool last_of(uint32_t *counter, uint32_t total) {
    __shared__ uint32_t done;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) {
        done = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        if (done == total - 1) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    const bool last = done == total - 1;
    __syncthreads();
    return last;
}

// Workgroups [0, quant_wgs) quantize x.  The others take a router row and 4 tokens
// each; the last of those tokens' workgroups makes their choices, and the last of all
// makes the plan.  With given choices there is one more workgroup, for the plan.
template <int WORDS>
__global__ __launch_bounds__(kThreads) void moe_prepare_kernel(MoeArgs a, int quant_wgs, int route, int plan) {
    if constexpr (WORDS > 0) {
        if (static_cast<int>(blockIdx.x) < quant_wgs) {
            const int t = static_cast<int>(blockIdx.x) * kThreads + threadIdx.x;
            const int blk = t / kQuantLanes, part = t % kQuantLanes;
            const int row = blk / a.sbk, b = blk - row * a.sbk;
            const bool valid = row < a.rows;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (valid && b < a.nbk)
                v = *reinterpret_cast<const float4 *>(a.x + static_cast<int64_t>(row) * a.k + b * kBlock + 4 * part);
            uint32_t h4, l4;
            const float s = quantize4<WORDS>(v, h4, l4);
            if (!valid) return;
            uint8_t *rec = a.xq + static_cast<int64_t>(row) * a.sbk * (WORDS * 32);
            *reinterpret_cast<uint32_t *>(rec + record_offset(a.tiled, WORDS, b, 0, part)) = h4;
            if (WORDS == 2) *reinterpret_cast<uint32_t *>(rec + record_offset(a.tiled, WORDS, b, 1, part)) = l4;
            if (part == 0) a.xs[blk] = s;
            return;
        }
    }
    if (route) {
        const int item = static_cast<int>(blockIdx.x) - quant_wgs;
        const int group = item / a.experts, t0 = group * kTokenGroup;
        route_logits(a, item - group * a.experts, t0);
        if (!last_of(a.counters + group * kMoeCounterStride, static_cast<uint32_t>(a.experts))) return;
        const int t = t0 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
        static_assert(kTokenGroup == kWaves, "a wave for each token");
        if (t < a.rows) {
            int id;
            float gate;
            choose(a, t, lane, id, gate);
            if (lane < a.top_k) {
                const int64_t at = static_cast<int64_t>(t) * a.top_k + lane;
                __hip_atomic_store(a.ids + at, id, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                __hip_atomic_store(a.gates + at, gate, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            if (plan && a.rows == 1) plan_one(a, lane, id, gate);
        }
        if (plan && a.rows == 1) return;
        const int groups = (a.rows + kTokenGroup - 1) / kTokenGroup;
        if (!plan) return;
        if (groups > 1) {
            if (!last_of(a.counters + kMoeSlice / kTokenGroup * kMoeCounterStride, static_cast<uint32_t>(groups))) return;
        } else {
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
        }
    }
    make_plan(a);
}

}  // namespace

hipError_t launch_moe(int mode, const MoeArgs &a, bool route, bool experts, hipStream_t stream) {
    const int quant_wgs =
        experts && mode != 0 ? (a.rows * a.sbk * kQuantLanes + kThreads - 1) / kThreads : 0;
    const int groups = (a.rows + kTokenGroup - 1) / kTokenGroup;
    const dim3 grid(quant_wgs + (route ? a.experts * groups : 1));
    if (mode == 2)
        moe_prepare_kernel<2><<<grid, kThreads, 0, stream>>>(a, quant_wgs, route, experts);
    else if (mode == 1)
        moe_prepare_kernel<1><<<grid, kThreads, 0, stream>>>(a, quant_wgs, route, experts);
    else
        moe_prepare_kernel<0><<<grid, kThreads, 0, stream>>>(a, quant_wgs, route, experts);
    if (hipError_t e = hipGetLastError(); e != hipSuccess || !experts) return e;
    return launch_moe_experts(mode, a, stream);
}

}  // namespace q8
