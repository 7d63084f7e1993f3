// sample.hip -- draws a token from each row of logits (temperature, top-k,
// top-p, min-p, a given random number).
//
// Mathematics.  With m the row's largest logit, token i has the integer weight
// w_i = floor(exp((l_i - m) / T) 2^44 + 1/2): exp in f64, then 44 bits after the
// point relative to the largest.  Integer sums are exact and do not depend on
// their order, so histograms filled with atomics, prefix sums and partial sums
// of any split agree to the last bit, call after call.  A token under 2^-45 of
// the largest has weight 0 and is never drawn.
//
// In descending order (ties: lowest index first) with running sums C_j, every
// filter keeps a prefix, and only the sum at its end matters:
//   top-k  : C_k;   top-p : P = the first C_j >= top_p C_k;   min-p : the sum of
//   weights >= min_p 2^44;   the kept total W is the smallest of the three, and
//   the token drawn is the first with C_j > u W (or C_j = W).
// So no full sort is needed: a histogram over x = (m - l) / T finds the bin that
// holds an end, and only that bin's tokens are gathered and sorted.
#include "sample.h"

#pragma clang fp contract(off)

namespace q8 {
namespace {

constexpr double kUnit = 17592186044416.0;  // 2^44
constexpr int kBins = 2048;
constexpr double kXRange = 31.25;           // weights are 0 beyond x = 45 ln 2 = 31.19
constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kList = 4096;                 // tokens one sort takes
constexpr int kMaxThreads = 256;            // of the maxima's workgroups
constexpr int kMaxPerThread = 4;            // float4 loads a thread of them makes

typedef unsigned long long u64;

struct __attribute__((packed, aligned(4))) Float4 {
    float v[4];
};

__device__ __forceinline__ float clean(float l) { return l == l ? l : -__builtin_inff(); }  // NaN: not a candidate

// Maxima of 64 consecutive logits: a thread takes four, 16 lanes meet.
__global__ __launch_bounds__(kMaxThreads) void sample_max_kernel(SampleArgs a) {
    const float *row = a.logits + static_cast<int64_t>(blockIdx.y) * a.ld;
#pragma unroll
    for (int p = 0; p < kMaxPerThread; ++p) {
        const int q = (static_cast<int>(blockIdx.x) * kMaxPerThread + p) * kMaxThreads + threadIdx.x;
        const int i = 4 * q;
        float v = -__builtin_inff();
        if (i + 4 <= a.n) {
            const Float4 f = *reinterpret_cast<const Float4 *>(row + i);
            v = fmaxf(fmaxf(clean(f.v[0]), clean(f.v[1])), fmaxf(clean(f.v[2]), clean(f.v[3])));
        } else {
            for (int j = i; j < a.n; ++j) v = fmaxf(v, clean(row[j]));
        }
#pragma unroll
        for (int off = 1; off < 16; off <<= 1) v = fmaxf(v, __shfl_xor(v, off, 64));
        const int sub = q / 16;
        if ((threadIdx.x & 15) == 0 && sub < a.nsub) a.submax[static_cast<int64_t>(blockIdx.y) * a.nsub + sub] = v;
    }
}

// Order-preserving key of a logit (equal values, -0 and +0 among them, have equal keys).
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

struct Row {
    const float *l;
    const float *submax;
    int n, nsub;
    float m;      // largest logit (> -inf)
    double rt;    // 1 / temperature
};

// x = (m - l) / T >= 0, infinite for tokens that are no candidates.
__device__ __forceinline__ double x_of(const Row &r, float l) {
    if (l == r.m) return 0.0;
    if (!(l > -__builtin_inff())) return __builtin_inf();
    return -((static_cast<double>(l) - static_cast<double>(r.m)) * r.rt);
}
__device__ __forceinline__ u64 weight_of(double x) {
    return x < kXRange ? static_cast<u64>(floor(exp(-x) * kUnit + 0.5)) : 0;
}
// Whether a token can be drawn (its weight is not 0).
__device__ __forceinline__ bool counts(double x) { return x < 31.0 || weight_of(x) > 0; }
__device__ __forceinline__ int bin_of(double x) {
    return x < kXRange ? min(kBins - 1, static_cast<int>(x * (kBins / kXRange))) : kBins;
}

struct Shared {
    u64 weight[kBins];
    uint32_t count[kBins];
    u64 list[kList];
    u64 wave[kWaves];
    uint32_t wave_c[kWaves];
    uint32_t fill;
    u64 pick_c, pick_w;
    uint32_t pick_at, pick_before;
};

// Inclusive prefix sums over the workgroup's threads of (v, c), in thread order.
__device__ __forceinline__ void block_scan(Shared &s, u64 &v, uint32_t &c) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const u64 ov = __shfl_up(v, off, 64);
        const uint32_t oc = __shfl_up(c, off, 64);
        if (lane >= off) {
            v += ov;
            c += oc;
        }
    }
    __syncthreads();
    if (lane == 63) {
        s.wave[wave] = v;
        s.wave_c[wave] = c;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        v += s.wave[w];
        c += s.wave_c[w];
    }
}

// A set of tokens next to each other in the descending order: those of bin `bin`
// of the histogram with keys in [klo, khi].  `above` and `above_c` are the
// weight and number of the tokens before it.
struct Span {
    int bin;
    uint32_t klo, khi;
    u64 above;
    uint32_t above_c;
    uint32_t count;
};

__device__ __forceinline__ bool in_span(const Row &r, const Span &sp, float l, double x) {
    if (bin_of(x) != sp.bin || !counts(x)) return false;
    const uint32_t k = key_of(l);
    return k >= sp.klo && k <= sp.khi;
}

// For every token of the row: f(index, logit).  Sub-blocks whose maximum the
// caller's `skip` rejects are not read.
template <typename S, typename F>
__device__ __forceinline__ void for_tokens(const Row &r, S skip, F f) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int b = wave; b < r.nsub; b += kWaves) {
        if (skip(r.submax[b])) continue;
        const int i = b * kSubBlock + lane;
        if (i < r.n) f(i, clean(r.l[i]));
    }
}

// Where a prefix ends: the first token, in descending order, whose running
// (sum, count) satisfies `cond` (monotone, true at the end of the span at the
// latest).  Results: its running sum, its own weight and its index.
struct End {
    u64 sum, weight;
    int32_t index;
};

template <typename C>
__device__ End find_end(Shared &s, const Row &r, Span sp, C cond) {
    while (true) {
        if (sp.count <= kList) {
            // gather, sort in descending (key, -index), scan
            __syncthreads();
            if (threadIdx.x == 0) s.fill = 0;
            uint32_t size = 64;
            while (size < sp.count) size <<= 1;
            for (uint32_t i = threadIdx.x; i < size; i += kThreads) s.list[i] = 0;
            __syncthreads();
            for_tokens(
                r, [&](float sub) { return bin_of(x_of(r, sub)) > sp.bin; },
                [&](int i, float l) {
                    if (!in_span(r, sp, l, x_of(r, l))) return;
                    const uint32_t at = atomicAdd(&s.fill, 1u);
                    if (at < kList) s.list[at] = (static_cast<u64>(key_of(l)) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
                });
            for (uint32_t k = 2; k <= size; k <<= 1)
                for (uint32_t j = k >> 1; j > 0; j >>= 1) {
                    __syncthreads();
                    for (uint32_t i = threadIdx.x; i < size / 2; i += kThreads) {
                        const uint32_t a = (i / j) * 2 * j + i % j, b = a + j;
                        const u64 va = s.list[a], vb = s.list[b];
                        if ((va < vb) == ((a & k) == 0)) {
                            s.list[a] = vb;
                            s.list[b] = va;
                        }
                    }
                }
            __syncthreads();
            constexpr int kPer = kList / kThreads;
            u64 w[kPer], own = 0;
            uint32_t own_c = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const uint32_t i = threadIdx.x * kPer + j;
                const bool ok = i < size && s.list[i] != 0;
                w[j] = ok ? weight_of(x_of(r, logit_of(static_cast<uint32_t>(s.list[i] >> 32)))) : 0;
                own += w[j];
                own_c += ok;
            }
            u64 run = own;
            uint32_t run_c = own_c;
            block_scan(s, run, run_c);
            run += sp.above - own;
            run_c += sp.above_c - own_c;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const uint32_t i = threadIdx.x * kPer + j;
                if (i >= size || s.list[i] == 0) continue;
                const bool before = run_c > sp.above_c && cond(run, run_c);
                run += w[j];
                ++run_c;
                if (!before && cond(run, run_c)) {
                    s.pick_c = run;
                    s.pick_w = w[j];
                    s.pick_at = 0xffffffffu - static_cast<uint32_t>(s.list[i]);
                }
            }
            __syncthreads();
            const End e{s.pick_c, s.pick_w, static_cast<int32_t>(s.pick_at)};
            __syncthreads();
            return e;
        }
        if (sp.klo == sp.khi) {
            // equal logits, in index order: the first number j with cond, then the j-th index
            const u64 w = weight_of(x_of(r, logit_of(sp.klo)));
            uint32_t lo = 1, hi = sp.count;
            while (lo < hi) {
                const uint32_t mid = (lo + hi) / 2;
                if (cond(sp.above + w * mid, sp.above_c + mid))
                    hi = mid;
                else
                    lo = mid + 1;
            }
            // count the ties of each thread's contiguous share of the row
            const int per = (r.n + kThreads - 1) / kThreads;
            const int i0 = min(r.n, static_cast<int>(threadIdx.x) * per), i1 = min(r.n, i0 + per);
            u64 none = 0;
            uint32_t c = 0;
            for (int i = i0; i < i1; ++i) c += key_of(clean(r.l[i])) == sp.klo;
            uint32_t run = c;
            block_scan(s, none, run);
            if (run >= lo && run - c < lo) {
                uint32_t left = lo - (run - c);
                int i = i0;
                for (; i < i1; ++i)
                    if (key_of(clean(r.l[i])) == sp.klo && --left == 0) break;
                s.pick_at = static_cast<uint32_t>(i);
            }
            __syncthreads();
            const End e{sp.above + w * lo, w, static_cast<int32_t>(s.pick_at)};
            __syncthreads();
            return e;
        }
        // too many tokens to sort: a histogram over the span's keys, largest first,
        // in the list's place (the bins' prefix sums stay)
        u64 *weight = s.list;
        uint32_t *count = reinterpret_cast<uint32_t *>(s.list + kBins);
        static_assert(kBins * 12 <= kList * 8, "the narrowing histogram fits the list");
        int shift = 0;
        while (((sp.khi - sp.klo) >> shift) >= kBins) ++shift;
        __syncthreads();
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            weight[i] = 0;
            count[i] = 0;
        }
        __syncthreads();
        for_tokens(
            r, [&](float sub) { return bin_of(x_of(r, sub)) > sp.bin; },
            [&](int i, float l) {
                const double x = x_of(r, l);
                if (!in_span(r, sp, l, x)) return;
                const uint32_t b = (sp.khi - key_of(l)) >> shift;
                atomicAdd(&weight[b], weight_of(x));
                atomicAdd(&count[b], 1u);
            });
        __syncthreads();
        const int b0 = 2 * threadIdx.x;
        const u64 w0 = weight[b0], w1 = weight[b0 + 1];
        const uint32_t c0 = count[b0], c1 = count[b0 + 1];
        u64 run = w0 + w1;
        uint32_t run_c = c0 + c1;
        block_scan(s, run, run_c);
        const u64 base = sp.above + run - w0 - w1;
        const uint32_t base_c = sp.above_c + run_c - c0 - c1;
        const bool at0 = base_c > sp.above_c && cond(base, base_c);
        const bool at1 = (base_c + c0 > sp.above_c) && cond(base + w0, base_c + c0);
        const bool at2 = (base_c + c0 + c1 > sp.above_c) && cond(base + w0 + w1, base_c + c0 + c1);
        if (!at0 && at1) {
            s.pick_at = b0;
            s.pick_c = base;
            s.pick_before = base_c;
            s.fill = c0;
        } else if (!at1 && at2) {
            s.pick_at = b0 + 1;
            s.pick_c = base + w0;
            s.pick_before = base_c + c0;
            s.fill = c1;
        }
        __syncthreads();
        const uint32_t b = s.pick_at;
        sp.above = s.pick_c;
        sp.above_c = s.pick_before;
        sp.count = s.fill;
        const uint32_t top = sp.khi - (b << shift);
        const uint32_t len = (1u << shift) - 1;
        sp.klo = top - min(len, top - sp.klo);
        sp.khi = top;
        __syncthreads();
    }
}

// One workgroup a row.
__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleArgs a) {
    __shared__ Shared s;
    const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    Row r;
    r.l = a.logits + static_cast<int64_t>(row) * a.ld;
    r.submax = a.submax + static_cast<int64_t>(row) * a.nsub;
    r.n = a.n;
    r.nsub = a.nsub;

    // the largest logit
    float m = -__builtin_inff();
    for (int b = tid; b < a.nsub; b += kThreads) m = fmaxf(m, r.submax[b]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    if (lane == 0) s.wave[wave] = __float_as_uint(m);
    if (tid == 0) s.pick_at = 0xffffffffu;
    __syncthreads();
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, __uint_as_float(static_cast<uint32_t>(s.wave[w])));
    r.m = m;
    if (!(m > -__builtin_inff())) {  // no candidate
        if (tid == 0) {
            a.idx[row] = -1;
            if (a.prob) a.prob[row] = 0.f;
        }
        return;
    }
    const float t = a.temperature ? a.temperature[row] : 1.0f;
    if (!(t > 0.0f)) {  // greedy: the lowest index among the largest
        for_tokens(
            r, [&](float sub) { return sub != m; }, [&](int i, float l) { if (l == m) atomicMin(&s.pick_at, static_cast<uint32_t>(i)); });
        __syncthreads();
        if (tid == 0) {
            a.idx[row] = static_cast<int32_t>(s.pick_at);
            if (a.prob) a.prob[row] = 1.f;
        }
        return;
    }
    r.rt = 1.0 / static_cast<double>(t);
    const int32_t top_k = a.top_k ? a.top_k[row] : 0;
    const float top_p = a.top_p ? a.top_p[row] : 1.f;
    const float min_p = a.min_p ? a.min_p[row] : 0.f;
    const double least = min_p > 0.f ? static_cast<double>(min_p) * kUnit : 0.0;

    // histogram of every token of non-zero weight, and the sum at or above min-p
    for (int i = tid; i < kBins; i += kThreads) {
        s.weight[i] = 0;
        s.count[i] = 0;
    }
    __syncthreads();
    u64 strong = 0;
    for_tokens(
        r, [&](float sub) { return !(x_of(r, sub) < kXRange); },
        [&](int, float l) {
            const double x = x_of(r, l);
            const u64 w = weight_of(x);
            if (w == 0) return;
            const int b = bin_of(x);
            atomicAdd(&s.weight[b], w);
            atomicAdd(&s.count[b], 1u);
            if (static_cast<double>(w) >= least) strong += w;
        });
    uint32_t zero = 0;
    block_scan(s, strong, zero);  // barriers: the histogram is complete
    if (tid == kThreads - 1) s.pick_c = strong;
    __syncthreads();
    u64 kept = s.pick_c;          // the sum that min-p keeps
    if (kept == 0) kept = static_cast<u64>(kUnit);
    __syncthreads();
    const int b0 = 2 * tid;
    u64 run = s.weight[b0] + s.weight[b0 + 1];
    uint32_t run_c = s.count[b0] + s.count[b0 + 1];
    block_scan(s, run, run_c);
    // inclusive prefixes in place
    const u64 w1 = s.weight[b0 + 1];
    const uint32_t c1 = s.count[b0 + 1];
    s.weight[b0 + 1] = run;
    s.weight[b0] = run - w1;
    s.count[b0 + 1] = run_c;
    s.count[b0] = run_c - c1;
    __syncthreads();

    // the span (one bin) in which `cond` becomes true
    auto bin_with = [&](auto cond) {
        const bool before = b0 > 0 && s.count[b0 - 1] > 0 && cond(s.weight[b0 - 1], s.count[b0 - 1]);
        const bool first = s.count[b0] > 0 && cond(s.weight[b0], s.count[b0]);
        const bool second = cond(s.weight[b0 + 1], s.count[b0 + 1]) && s.count[b0 + 1] > 0;
        if (!before && first)
            s.pick_at = b0;
        else if (!first && second)
            s.pick_at = b0 + 1;
        __syncthreads();
        const int b = static_cast<int>(s.pick_at);
        Span sp;
        sp.bin = b;
        sp.klo = 0;
        sp.khi = 0xffffffffu;
        sp.above = b > 0 ? s.weight[b - 1] : 0;
        sp.above_c = b > 0 ? s.count[b - 1] : 0;
        sp.count = s.count[b] - sp.above_c;
        __syncthreads();
        return sp;
    };
    const u64 all = s.weight[kBins - 1];
    const uint32_t all_c = s.count[kBins - 1];
    u64 limit = all;  // C_k
    if (top_k > 0 && static_cast<uint32_t>(top_k) < all_c) {
        const uint32_t k = static_cast<uint32_t>(top_k);
        auto cond = [=](u64, uint32_t c) { return c >= k; };
        limit = find_end(s, r, bin_with(cond), cond).sum;
    }
    if (top_p < 1.f) {
        const double target = static_cast<double>(top_p) * static_cast<double>(limit);
        auto cond = [=](u64 c, uint32_t) { return static_cast<double>(c) >= target; };
        limit = find_end(s, r, bin_with(cond), cond).sum;
    }
    if (limit < kept) kept = limit;
    const double target = static_cast<double>(a.u[row]) * static_cast<double>(kept);
    auto cond = [=](u64 c, uint32_t) { return static_cast<double>(c) > target || c >= kept; };
    const End e = find_end(s, r, bin_with(cond), cond);
    if (tid == 0) {
        a.idx[row] = e.index;
        if (a.prob) a.prob[row] = static_cast<float>(static_cast<double>(e.weight) / static_cast<double>(kept));
    }
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, hipStream_t stream) {
    const int per = kMaxThreads * kMaxPerThread * 4;
    sample_max_kernel<<<dim3((a.n + per - 1) / per, a.rows), kMaxThreads, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    sample_row_kernel<<<dim3(a.rows), kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace q8
