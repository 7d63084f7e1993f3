// sample.hip -- draws a token from each row of logits (temperature, top-k,
// top-p, min-p, a given random number).
//
// Mathematics.  With m the row's largest logit, token i has the integer weight
// w_i = exp((l_i - m) / T) 2^44, in f64, rounded to a whole number: 44 bits after the
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
// So no full sort is needed.
//
// Kernels.  The first reads the logits once and leaves the maximum of every 64.
// The second has two ways through a row:
//  - few tokens matter (top-k up to 512, or min-p alone): the maxima bound the
//    tokens in question from below (the k-th largest maximum has k tokens at or
//    above it), only the sub-blocks that can hold one are read again, and one
//    workgroup sorts and scans the few tokens found;
//  - else a histogram of the weights over x = (m - l) / T, filled by one or more
//    workgroups a row, tells which bin holds each end; the third kernel gathers and
//    sorts just those bins' tokens.
// A row is read from memory once; the caches serve what is read again.
//
// Bound.  The chain of dependent steps, and with many rows one workgroup's share of a row:
// one row of 151936 with top-k 3 + 10 + 2 us; 8 rows of 32003 with top-p 3 + 11 + 18 us; 64
// rows of 151936, each kind of filter, 8 + 22 + 30 us (39 MB), all with top-p 8 + 24 + 35; 256
// rows of 50257, min-p on half, 9 + 28 + 21 us (51 MB), all plain 8 + 24 + 24.  The histogram
// of 64 rows takes as long for 24 rows of them as for all: workgroups are dealt by the
// number of rows, so 96 and 128 of 256 CUs work in the first of each pair, and what counts is
// the time of one workgroup (41000 and 50000 logits; some 35 instructions each, most of
// them f64, are 9 and 11 us of a CU, the rest is latency).
#include "device.h"
#include "sample.h"

#pragma clang fp contract(off)

namespace q8 {
namespace {

constexpr double kUnit = 17592186044416.0;  // 2^44
constexpr int kBins = kSampleBins;
constexpr double kXLast = 31.191623125197536;  // 45 ln 2: weights are 0 beyond
// Bins of the histogram over x = (m - l) / T: narrow ones up to 16, where the ends of the
// prefixes are as good as always (of 2^19 equal tokens there the weight is 6 %), wider
// ones behind.  With equal bins, 66 a unit, the tokens of a top-p's end and of the draw
// could be more than one draw takes (152000 tokens, T = 1.4: 130 us a call, not 60).
constexpr double kXFine = 16.0, kFinePerX = 112.0, kCoarsePerX = 16.75;
constexpr double kFineBins = kXFine * kFinePerX;
static_assert(kFineBins + (kXLast - kXFine) * kCoarsePerX < kBins - 1.5, "no token is in the last bin");
constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr int kList = 4096;                 // tokens one sort takes
constexpr int kQuick = kNear;               // tokens one draw takes: one a thread
static_assert(kNear == kThreads, "one token a thread");
constexpr int kQuickTopK = 512;
constexpr int kMaxSubs = static_cast<int>((kSampleMaxN + kSubBlock - 1) / kSubBlock);
constexpr int kSubsPerThread = (kMaxSubs + kThreads - 1) / kThreads;
constexpr int kMaxThreads = 256;            // of the maxima's workgroups
constexpr int kMaxPerThread = 4;            // float4 loads a thread of them makes
static_assert(kMaxWgLogits == kMaxThreads * kMaxPerThread * 4 && kMaxThreads == 256, "nwave counts these");

typedef unsigned long long u64;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float clean(float l) { return l == l ? l : -__builtin_inff(); }  // NaN: not a candidate

// Up to four consecutive logits: those of [first, end) among row[at .. at + 3].  The
// load is the same for every lane, with no branch around it (lanes at the end of the
// row step back), so that several can be in flight; trim() makes the others -inf.
struct Quad {
    float v[4];
    int at, first, end;
    __device__ __forceinline__ void trim() {
        if (first + 4 > end) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (at + j < first || at + j >= end) v[j] = -__builtin_inff();
        }
    }
};

// A row of logits as a range-checked buffer (its loads need dword alignment only).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t row_buffer(const SampleArgs &a, int row) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(a.logits + static_cast<int64_t>(row) * a.ld), 0, a.n * 4,
                                             0x00020000);
}
__device__ __forceinline__ float load1(__amdgpu_buffer_rsrc_t row, int i) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(row, 4 * i, 0, 0));
}

__device__ __forceinline__ Quad load4(__amdgpu_buffer_rsrc_t row, int i, int end, int n) {
    Quad q;
    q.first = i;
    q.end = end;
    q.at = max(min(i, n - 4), 0);
    if (n >= 4) {  // the same for the whole launch
        const u32x4 d = __builtin_amdgcn_raw_buffer_load_b128(row, 4 * q.at, 0, 0);
        q.v[0] = __uint_as_float(d.x);
        q.v[1] = __uint_as_float(d.y);
        q.v[2] = __uint_as_float(d.z);
        q.v[3] = __uint_as_float(d.w);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) q.v[j] = load1(row, min(j, n - 1));
    }
    return q;
}

// A row's parameters, and which way it goes.
struct Params {
    float t;
    int32_t top_k;  // 0: all
    float top_p;    // 1: all
    float min_p;
    u64 least;      // smallest weight that min-p keeps, 0: all
    float u;
    bool greedy, by_k, by_p;  // the quick ways: the largest logit; few tokens, by top-k or by min-p
    __device__ __forceinline__ bool quick() const { return greedy || by_k || by_p; }
};

__device__ __forceinline__ Params params_of(const SampleArgs &a, int row) {
    Params p;
    p.t = a.temperature ? a.temperature[row] : 1.0f;
    p.top_k = a.top_k ? max(a.top_k[row], 0) : 0;
    if (p.top_k >= a.n) p.top_k = 0;
    p.top_p = a.top_p ? a.top_p[row] : 1.f;
    p.min_p = a.min_p ? a.min_p[row] : 0.f;
    // w >= min_p 2^44 for whole w; beyond 2^45 there is no such weight
    p.least = p.min_p > 0.f ? static_cast<u64>(ceil(fmin(static_cast<double>(p.min_p) * kUnit, 2.0 * kUnit))) : 0;
    p.u = a.u[row];
    p.greedy = !(p.t > 0.0f);
    p.by_k = p.top_k > 0 && p.top_k <= min(kQuickTopK, a.nsub);
    p.by_p = !p.greedy && p.top_k == 0 && !(p.top_p < 1.f) && p.min_p > 0.f;
    return p;
}

// Maxima of 64 consecutive logits (a thread takes four, 16 lanes meet) and of every
// wave's 1024.
__global__ __launch_bounds__(kMaxThreads) void sample_max_kernel(SampleArgs a) {
    const __amdgpu_buffer_rsrc_t row = row_buffer(a, blockIdx.x);
    const int q0 = static_cast<int>(blockIdx.y) * kMaxPerThread * kMaxThreads + threadIdx.x;
    Quad f[kMaxPerThread];
#pragma unroll
    for (int p = 0; p < kMaxPerThread; ++p) f[p] = load4(row, min(4 * (q0 + p * kMaxThreads), a.n), a.n, a.n);
    if (blockIdx.y == 0 && threadIdx.x == 0) a.state[blockIdx.x] = RowState{0, 0, 0, 0};
    float most = -__builtin_inff();
#pragma unroll
    for (int p = 0; p < kMaxPerThread; ++p) {
        f[p].trim();
        // fmaxf passes a signaling NaN on and drops a quiet one: the sums are quiet, so that NaN
        // loses every comparison
        const float v = row_max(fmaxf(fmaxf(f[p].v[0] + 0.0f, f[p].v[1] + 0.0f), fmaxf(f[p].v[2] + 0.0f, f[p].v[3] + 0.0f)));
        most = fmaxf(most, v);
        const int sub = (q0 + p * kMaxThreads) / 16;
        if ((threadIdx.x & 15) == 0 && sub < a.nsub) a.submax[static_cast<int64_t>(blockIdx.x) * a.nsub + sub] = v;
    }
    most = wave_max(most);
    if ((threadIdx.x & 63) == 0)
        a.wavemax[static_cast<int64_t>(blockIdx.x) * a.nwave + blockIdx.y * (kMaxThreads / 64) + threadIdx.x / 64] = most;
}

// Order-preserving key of a logit (equal values, -0 and +0 among them, have equal keys).
__device__ __forceinline__ uint32_t key_of(float l) {
    const uint32_t b = __float_as_uint(l + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}
// Sort key of a token: larger logits first, then smaller indices; never 0.
__device__ __forceinline__ u64 token_of(float l, int i) {
    return (static_cast<u64>(key_of(l)) << 32) | (0xffffffffu - static_cast<uint32_t>(i));
}

struct Row {
    __amdgpu_buffer_rsrc_t l;
    int n, nsub;
    float m;      // largest logit (> -inf)
    double m64;
    bool infinite;  // m is +inf
    double rt;    // 1 / temperature
};

// x = (m - l) / T >= 0 (infinite or NaN for tokens that are no candidates).
__device__ __forceinline__ double x_of(const Row &r, float l) {
    if (r.infinite) return l == r.m ? 0.0 : __builtin_inf();  // the same for the whole row
    return (r.m64 - static_cast<double>(l)) * r.rt;
}

// exp(-x) 2^44 rounded to a whole number, for 0 <= x <= kXLast.  -x = k ln 2 + t with
// |t| <= ln 2 / 2 (k out of the mantissa of a sum with 3 * 2^51); exp(t) by the
// polynomial of degree 10 that meets it at the 11 Chebyshev points of that interval
// (relative error 2^-51.4, exact at 0); 2^(k + 44) goes into the exponent, and the
// whole number is read out of the mantissa of a sum with 2^52.
__device__ __forceinline__ u64 weight_within(double x) {
    constexpr double kShift = 6755399441055744.0;
    const double y = __builtin_fma(x, -1.4426950408889634, kShift);
    const uint32_t k = static_cast<uint32_t>(__builtin_bit_cast(u64, y));
    const double t = __builtin_fma(y - kShift, -0.69314718055994529, -x);
    double p = 2.762635725527078e-07;
    p = __builtin_fma(p, t, 2.7640180812804505e-06);
    p = __builtin_fma(p, t, 2.480150434696448e-05);
    p = __builtin_fma(p, t, 0.00019841170270400204);
    p = __builtin_fma(p, t, 0.0013888888932488625);
    p = __builtin_fma(p, t, 0.008333333385667814);
    p = __builtin_fma(p, t, 0.04166666666657314);
    p = __builtin_fma(p, t, 0.16666666666554406);
    p = __builtin_fma(p, t, 0.5000000000000006);
    p = __builtin_fma(p, t, 1.0000000000000067);
    p = __builtin_fma(p, t, 1.0);
    const u64 bits = __builtin_bit_cast(u64, p);
    const uint32_t high = static_cast<uint32_t>(bits >> 32) + ((k + 44) << 20);
    const double v = __builtin_bit_cast(double, (static_cast<u64>(high) << 32) | static_cast<uint32_t>(bits));
    return __builtin_bit_cast(u64, v + 4503599627370496.0) & 0xfffffffffffffull;
}
// Where x is among the bins (bin b is around position b), and the x of a position.
__device__ __forceinline__ double bin_position(double x) {
    return fmin(x * kFinePerX, __builtin_fma(x, kCoarsePerX, kFineBins - kXFine * kCoarsePerX));
}
__device__ __forceinline__ double x_at(double position) {
    return fmax(position / kFinePerX, kXFine + (position - kFineBins) / kCoarsePerX);
}
// The nearest bin's number, for 0 <= x <= kXLast.
__device__ __forceinline__ int bin_within(double x) {
    return static_cast<int>(static_cast<uint32_t>(__builtin_bit_cast(u64, bin_position(x) + 4503599627370496.0)));
}
__device__ __forceinline__ u64 weight_of(double x) { return x <= kXLast ? weight_within(x) : 0; }
// Bin of a token that can be drawn; kBins for the others.
__device__ __forceinline__ int bin_of(double x) {
    return x <= kXLast ? bin_within(x) : kBins;
}

struct Shared {
    u64 weight[kBins];       // histogram, then its prefix sums
    uint32_t count[kBins];
    u64 list[kList];         // tokens
    uint16_t subs[kMaxSubs]; // sub-blocks to read
    u64 wave[kWaves];
    uint32_t wave_c[kWaves];
    uint32_t fill, nsubs;
    u64 pick_c, pick_w;
    uint32_t pick_at, pick_before;
};

template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t dpp_or0(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, true));
}
template <int CTRL, int ROWS>
__device__ __forceinline__ void scan_step(u64 &v, uint32_t &c) {
    const u64 lo = dpp_or0<CTRL, ROWS>(static_cast<uint32_t>(v)), hi = dpp_or0<CTRL, ROWS>(static_cast<uint32_t>(v >> 32));
    c += dpp_or0<CTRL, ROWS>(c);
    v += (hi << 32) | lo;
}

// Inclusive prefix sums over the workgroup's threads of (v, c), in thread order.
__device__ __forceinline__ void block_scan(Shared &s, u64 &v, uint32_t &c) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    scan_step<0x111, 0xf>(v, c);  // row_shr 1, 2, 4, 8: within 16 lanes
    scan_step<0x112, 0xf>(v, c);
    scan_step<0x114, 0xf>(v, c);
    scan_step<0x118, 0xf>(v, c);
    scan_step<0x142, 0xa>(v, c);  // lane 15 of rows 0, 2 to rows 1, 3
    scan_step<0x143, 0xc>(v, c);  // lane 31 to rows 2, 3
    __syncthreads();
    if (lane == 63) {
        s.wave[wave] = v;
        s.wave_c[wave] = c;
    }
    __syncthreads();
#pragma clang loop unroll(disable)
    for (int w = 0; w < wave; ++w) {
        v += s.wave[w];
        c += s.wave_c[w];
    }
}

// This thread's share of a row's sub-block maxima: those of sub-blocks
// tid, tid + 1024, ..
struct Subs {
    float v[kSubsPerThread];
};

__device__ __forceinline__ Subs load_subs(const SampleArgs &a, int row) {
    const float *submax = a.submax + static_cast<int64_t>(row) * a.nsub;
    Subs m;
#pragma unroll
    for (int q = 0; q < kSubsPerThread; ++q) {
        m.v[q] = -__builtin_inff();
        if (q * kThreads >= a.nsub) break;
        const int b = q * kThreads + static_cast<int>(threadIdx.x);
        const float v = submax[min(b, a.nsub - 1)];
        m.v[q] = b < a.nsub ? v : -__builtin_inff();
    }
    return m;
}

// For every token of the sub-blocks whose maximum `want` takes: f(index, logit), four
// at a time where `some` finds one of the four in question (with -inf and any index
// where there is no token).  One workgroup may look through a whole row here, and
// what bounds that is the arithmetic on each token: `some` is all that most cost.
// The sub-blocks are listed first (one LDS atomic a wave), so that a thread has
// several loads in flight.  Of `parts` (a power of two) workgroups, this one takes
// every parts-th sub-block.
template <int kAhead, typename S, typename Q, typename F>
__device__ __forceinline__ void for_tokens(Shared &s, const Row &r, const Subs &subs, S want, Q some, F f, int parts = 1,
                                           int part_at = 0) {
    constexpr int kGroups = kThreads / 16;
    // opaque, so that nothing computed from them here is kept in registers between
    // the calls of this function (the kernel then spilled)
    uint32_t tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    __syncthreads();
    if (tid == 0) s.nsubs = 0;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSubsPerThread; ++q) {
        if (q * kThreads >= r.nsub) break;
        const int b = q * kThreads + static_cast<int>(tid);
        float sub = subs.v[q];
        asm volatile("" : "+v"(sub));
        const bool yes = b < r.nsub && (b & (parts - 1)) == part_at && want(sub);
        const u64 set = __ballot(yes);
        if (set) {
            uint32_t at = 0;
            if ((tid & 63) == 0) at = atomicAdd(&s.nsubs, static_cast<uint32_t>(__popcll(set)));
            at = __builtin_amdgcn_readfirstlane(at);
            if (yes) s.subs[at + __popcll(set & ((1ull << (tid & 63)) - 1))] = static_cast<uint16_t>(b);
        }
    }
    __syncthreads();
    const int total = static_cast<int>(s.nsubs), part = 4 * (tid & 15);
#pragma clang loop unroll(disable)
    for (int g = static_cast<int>(tid / 16); g < total; g += kGroups * kAhead) {
        Quad v[kAhead];
        int at[kAhead];
#pragma unroll
        for (int p = 0; p < kAhead; ++p) at[p] = s.subs[min(g + p * kGroups, total - 1)];
#pragma unroll
        for (int p = 0; p < kAhead; ++p)
            v[p] = load4(r.l, g + p * kGroups < total ? min(at[p] * kSubBlock + part, r.n) : r.n, r.n, r.n);
#pragma unroll
        for (int p = 0; p < kAhead; ++p) {
            if (!some(v[p].v)) continue;
            v[p].trim();
#pragma unroll
            for (int j = 0; j < 4; ++j) f(v[p].at + j, v[p].v[j]);
        }
    }
}

// A logit at or below every logit of bins 0 .. b: m - T x of its lower edge, lowered
// well past the rounding.  Infinite where that is no number.
__device__ __forceinline__ float bin_floor(const Row &r, int b) {
    const double m = static_cast<double>(r.m), down = x_at(b + 0.5) / r.rt;
    const float f = static_cast<float>(m - down - (1e-6 * (fabs(m) + down) + 1e-30));
    return f == f ? f : -__builtin_inff();
}

// Likewise at or above every logit of bins b and on.
__device__ __forceinline__ float bin_ceil(const Row &r, int b) {
    const double m = static_cast<double>(r.m), down = x_at(b - 0.5) / r.rt;
    const float f = static_cast<float>(m - down + (1e-6 * (fabs(m) + down) + 1e-30));
    return b > 0 && f == f ? f : __builtin_inff();
}

// A set of tokens next to each other in the descending order: those of bin `bin`
// of the histogram with keys in [klo, khi].  `above` is the weight before it.
// No logit of it is under llo: a cheap test before the exact one.
struct Span {
    int bin;
    uint32_t klo, khi;
    float llo;
    u64 above;
    uint32_t above_c;  // tokens before it (kept only where a top-k needs them)
    uint32_t count;    // tokens in it, or a bound above their number
};

__device__ __forceinline__ bool in_span(const Row &r, const Span &sp, float l) {
    if (!(l >= sp.llo)) return false;
    const double x = x_of(r, l);
    if (bin_of(x) != sp.bin) return false;
    const uint32_t k = key_of(l);
    return k >= sp.klo && k <= sp.khi;
}

// Where a prefix ends: the first token, in descending order, whose running
// (sum, count) satisfies `cond` (monotone, true at the end of the span at the
// latest).  Results: its running sum, its own weight and its index.
struct End {
    u64 sum, weight;
    int32_t index;
};

// Sorts the first `size` (a power of two) entries of the list, descending.
__device__ __forceinline__ void sort_list(Shared &s, uint32_t size) {
#pragma clang loop unroll(disable)
    for (uint32_t k = 2; k <= size; k <<= 1)
#pragma clang loop unroll(disable)
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
}

// The workgroup's values (one a thread, `size` of them: a power of two from 64 to
// 1024), sorted in descending order through `buf`.  Exchanges of up to 32 places
// stay inside a wave; the others go through LDS.
__device__ __forceinline__ u64 sort_one_a_thread(u64 v, u64 *buf, uint32_t size) {
    const uint32_t i = threadIdx.x;
#pragma clang loop unroll(disable)
    for (uint32_t k = 2; k <= size; k <<= 1) {
#pragma clang loop unroll(disable)
        for (uint32_t j = k >> 1; j > 0; j >>= 1) {
            u64 o;
            if (j >= 64) {
                __syncthreads();
                buf[i] = v;
                __syncthreads();
                o = buf[i ^ j];
            } else {
                o = __shfl_xor(v, static_cast<int>(j), 64);
            }
            const bool largest = ((i & j) == 0) == ((i & k) == 0);
            v = largest == (o > v) ? o : v;
        }
    }
    __syncthreads();
    return v;
}

// When a prefix has ended: at a number of tokens (kind 0), at a sum of at least
// `target` (1), or at a sum over `target` or of `total` (2).
struct EndTest {
    int kind;
    uint32_t number;
    double target;
    u64 total;
    __device__ __forceinline__ bool operator()(u64 sum, uint32_t count) const {
        if (kind == 0) return count >= number;
        const double c = static_cast<double>(sum);
        return kind == 1 ? c >= target : c > target || sum >= total;
    }
};

__device__ __forceinline__ End find_end(Shared &s, const Row &r, const Subs &subs, Span sp, const EndTest &cond) {
    const auto want = [&](float sub) { return sub >= sp.llo && bin_of(x_of(r, sub)) <= sp.bin; };
    const auto some = [&](const float *v) { return v[0] >= sp.llo || v[1] >= sp.llo || v[2] >= sp.llo || v[3] >= sp.llo; };
    while (true) {
        if (sp.count <= kList) {
            // gather, sort in descending (key, -index), scan
            __syncthreads();
            if (threadIdx.x == 0) s.fill = 0;
            for_tokens<1>(s, r, subs, want, some, [&](int i, float l) {
                if (!in_span(r, sp, l)) return;
                const uint32_t at = atomicAdd(&s.fill, 1u);
                if (at < kList) s.list[at] = token_of(l, i);
            });
            __syncthreads();
            const uint32_t fill = min(s.fill, static_cast<uint32_t>(kList));
            uint32_t size = 64;
            while (size < fill) size <<= 1;
            for (uint32_t i = fill + threadIdx.x; i < size; i += kThreads) s.list[i] = 0;
            sort_list(s, size);
            constexpr int kPer = kList / kThreads;
            u64 w[kPer], own = 0;
            uint32_t own_c = 0;
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const uint32_t i = threadIdx.x * kPer + j;
                const bool ok = i < fill;
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
                if (i >= fill) continue;
                const bool before = i > 0 && cond(run, run_c);
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
#pragma clang loop unroll(disable)
            for (int i = i0; i < i1; ++i) c += key_of(clean(load1(r.l, i))) == sp.klo;
            uint32_t run = c;
            block_scan(s, none, run);
            if (run >= lo && run - c < lo) {
                uint32_t left = lo - (run - c);
                int i = i0;
                for (; i < i1; ++i)
                    if (key_of(clean(load1(r.l, i))) == sp.klo && --left == 0) break;
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
#pragma clang loop unroll(disable)
        for (int i = threadIdx.x; i < kBins; i += kThreads) {
            weight[i] = 0;
            count[i] = 0;
        }
        for_tokens<1>(s, r, subs, want, some, [&](int, float l) {
            if (!in_span(r, sp, l)) return;
            const uint32_t b = (sp.khi - key_of(l)) >> shift;
            atomicAdd(&weight[b], weight_of(x_of(r, l)));
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

__device__ __forceinline__ void write_row(const SampleArgs &a, int row, int32_t idx, float prob) {
    a.idx[row] = idx;
    if (a.prob) a.prob[row] = prob;
}

__device__ __forceinline__ void write_draw(const SampleArgs &a, int row, int32_t idx, u64 weight, u64 kept) {
    write_row(a, row, idx, static_cast<float>(static_cast<double>(weight) / static_cast<double>(kept)));
}

// What a call of draw_from knows when it starts.
struct Known {
    bool bins;     // the histogram's prefix sums are there, and the list holds whole bins
    u64 limit;     // C_k where top-k is off (bins)
    u64 strong;    // the sum that min-p keeps (bins)
};

// Ranges of bins, and windows of logits that hold them.
struct Ranges {
    int first[3], last[3];
    float lo[3], hi[3];
};

// Lists the tokens in the windows (a superset of the ranges' tokens, but for the
// rounding of their limits) in s.list; returns their number, of which only the first
// kQuick are there.
__device__ __forceinline__ uint32_t gather(Shared &s, const Row &r, const Subs &subs, const Ranges &g, int parts,
                                           int part_at) {
    if (threadIdx.x == 0) s.fill = 0;  // for_tokens begins with a barrier
    const float least = fminf(fminf(g.lo[0], g.lo[1]), g.lo[2]);
    const bool two = g.first[1] <= g.last[1], three = g.first[2] <= g.last[2];
    // a window as |l - mid| <= half: one subtraction a token, and one comparison for four
    float mid[3], half[3];
#pragma unroll
    for (int w = 0; w < 3; ++w) {
        const float hi = fminf(g.hi[w], r.m);
        mid[w] = 0.5f * g.lo[w] + 0.5f * hi;
        half[w] = (0.5f * hi - 0.5f * g.lo[w]) + 1e-6f * (fabsf(hi) + fabsf(g.lo[w]));
        if (!(fabsf(mid[w]) < __builtin_inff()) || !(half[w] < __builtin_inff())) {
            mid[w] = 0.f;
            half[w] = __builtin_inff();
        }
    }
    const auto near_to = [&](const float *v, int w) {
        const float d0 = fabsf(v[0] - mid[w]), d1 = fabsf(v[1] - mid[w]), d2 = fabsf(v[2] - mid[w]), d3 = fabsf(v[3] - mid[w]);
        return fminf(fminf(d0, d1), fminf(d2, d3)) <= half[w];
    };
    for_tokens<4>(
        s, r, subs, [&](float sub) { return sub >= least; },
        [&](const float *v) { return near_to(v, 0) || (two && near_to(v, 1)) || (three && near_to(v, 2)); },
        [&](int i, float l) {
            bool in = l >= g.lo[0] && l <= g.hi[0];
            if (two) in = in || (l >= g.lo[1] && l <= g.hi[1]);  // the same for the workgroup
            if (three) in = in || (l >= g.lo[2] && l <= g.hi[2]);
            if (!in || !(l > -__builtin_inff())) return;
            const uint32_t at = atomicAdd(&s.fill, 1u);
            if (at < kQuick) s.list[at] = token_of(l, i);
        },
        parts, part_at);
    __syncthreads();
    return s.fill;
}

// Sorts the listed tokens (`near` of them, at most one a thread) and draws.  Without
// `bins` the only range is a prefix of the order that holds the end of every filter;
// with it the ranges are the bins that can hold those ends, and a token's running sum
// is its bin's prefix sum plus what precedes it in its bin.
__device__ __forceinline__ void draw_from(Shared &s, const SampleArgs &a, const Row &r, const Params &p, int row,
                                          const Ranges &g, const Known &known, int near) {
    const int tid = threadIdx.x;
    // those of the ranges themselves; the others become 0 and go last
    u64 in = tid < near ? s.list[tid] : 0;
    if (in) {
        const int b = bin_of(x_of(r, logit_of(static_cast<uint32_t>(in >> 32))));
        const bool yes = (b >= g.first[0] && b <= g.last[0]) || (b >= g.first[1] && b <= g.last[1]) ||
                         (b >= g.first[2] && b <= g.last[2]);
        if (!yes) s.list[tid] = in = 0;
    }
    if (tid == 0) s.nsubs = 0;
    __syncthreads();
    const u64 set = __ballot(in != 0);
    if ((tid & 63) == 0 && set) atomicAdd(&s.nsubs, static_cast<uint32_t>(__popcll(set)));
    __syncthreads();
    const int fill = static_cast<int>(s.nsubs);
    u64 *sorted = s.list + kQuick;
    if (near <= 128) {
        // rank of a token = tokens before it; 8 or 16 threads share one
        const int parts = near <= 64 ? 16 : 8;
        const int e = tid / parts;
        const u64 mine = e < near ? s.list[e] : 0;
        int rank = 0;
        if (mine)
#pragma clang loop unroll(disable)
            for (int j = tid % parts; j < near; j += parts) rank += s.list[j] > mine;
        for (int off = 1; off < parts; off <<= 1) rank += __shfl_xor(rank, off, 64);
        if (mine && tid % parts == 0) sorted[rank] = mine;
    } else {
        uint32_t size = 256;
        while (size < static_cast<uint32_t>(near)) size <<= 1;
        const u64 v = sort_one_a_thread(tid < near ? s.list[tid] : 0, s.list + 2 * kQuick, size);
        sorted[tid] = v;
    }
    __syncthreads();
    const u64 token = tid < fill ? sorted[tid] : 0;
    const double x = token ? x_of(r, logit_of(static_cast<uint32_t>(token >> 32))) : __builtin_inf();
    const u64 w = weight_of(x);
    u64 run = w;
    uint32_t number = tid + 1, none = 0;  // of the token in the order
    block_scan(s, run, none);
    if (known.bins) {
        u64 *start = reinterpret_cast<u64 *>(s.subs);                        // list sums at the bins' first tokens
        uint32_t *start_at = reinterpret_cast<uint32_t *>(s.list + 2 * kQuick);  // and their places
        static_assert(sizeof(s.subs) >= sizeof(u64) * kBins && 2 * kQuick * 8 + kBins * 4 <= kList * 8, "room for them");
        const int b = token ? bin_of(x) : kBins;
        const u64 prev = token && tid > 0 ? sorted[tid - 1] : 0;
        if (token && !(prev && bin_of(x_of(r, logit_of(static_cast<uint32_t>(prev >> 32)))) == b)) {
            start[b] = run - w;
            start_at[b] = tid;
        }
        __syncthreads();
        if (token) {
            run += (b > 0 ? s.weight[b - 1] : 0) - start[b];
            number += (b > 0 ? s.count[b - 1] : 0) - start_at[b];
        }
    }
    const u64 before = run - w;
    // C_k, then the end of top-p, then of min-p; each found by the one thread it ends at
    if (tid == 0) {
        s.pick_c = known.limit;
        s.pick_w = known.bins ? known.strong : static_cast<u64>(kUnit);  // min-p keeps one token at least
    }
    __syncthreads();
    if (token && p.top_k > 0 && number == static_cast<uint32_t>(p.top_k)) s.pick_c = run;
    if (!known.bins) {
        if (tid == fill - 1 && (p.top_k == 0 || p.top_k > fill)) s.pick_c = run;
        if (token && (p.least == 0 ? tid == fill - 1 : w >= p.least)) atomicMax(&s.pick_w, run);
    }
    __syncthreads();
    const double target = static_cast<double>(p.top_p) * static_cast<double>(s.pick_c);
    __syncthreads();
    if (p.top_p < 1.f && token && static_cast<double>(run) >= target && !(before > 0 && static_cast<double>(before) >= target))
        s.pick_c = run;
    __syncthreads();
    const u64 kept = s.pick_c < s.pick_w ? s.pick_c : s.pick_w;
    const double at = static_cast<double>(p.u) * static_cast<double>(kept);
    auto cond = [&](u64 c) { return static_cast<double>(c) > at || c >= kept; };
    if (token && cond(run) && !(before > 0 && cond(before)))
        write_draw(a, row, static_cast<int32_t>(0xffffffffu - static_cast<uint32_t>(token)), w, kept);
}

// Adds the tokens of [i0, i1) to the histogram in LDS; returns this thread's part
// of the weights that min-p keeps.  `tail`: from this bin on, tokens lie behind
// every end that is looked for, and only their sum matters: they go to the last
// bin (which no token has) in one piece.  What bounds this is the f64 arithmetic,
// about 20 operations a token; four tokens go side by side without branches (with
// a branch for each the chains ran one after the other, three times slower).
__device__ __forceinline__ u64 add_tokens(Shared &s, const Row &r, const Params &p, int i0, int i1, int tail) {
    u64 strong = 0, rest = 0;
    constexpr int kAhead = 4, kStride = 4 * kThreads;
    int i = i0 + 4 * static_cast<int>(threadIdx.x);
    Quad next[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) next[q] = load4(r.l, min(i + q * kStride, i1), i1, r.n);
#pragma clang loop unroll(disable)
    for (; i < i1; i += kStride) {
        Quad v = next[0];
#pragma unroll
        for (int q = 0; q + 1 < kAhead; ++q) next[q] = next[q + 1];
        next[kAhead - 1] = load4(r.l, min(i + kAhead * kStride, i1), i1, r.n);
        v.trim();
        double x[4];
        u64 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = x_of(r, v.v[j]);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = weight_within(x[j]);
        if (p.least > 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) strong += x[j] <= kXLast && w[j] >= p.least ? w[j] : 0;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int b = bin_within(x[j]);
            if (x[j] <= kXLast) {
                if (b >= tail) {
                    rest += w[j];
                } else {
                    atomicAdd(&s.weight[b], w[j]);
                    if (p.top_k > 0) atomicAdd(&s.count[b], 1u);
                }
            }
        }
    }
    if (rest) atomicAdd(&s.weight[kBins - 1], rest);
    return strong;
}

// The row's largest logit, to every thread.
__device__ __forceinline__ float largest(Shared &s, const SampleArgs &a, int row) {
    static_assert(kSampleMaxN / 1024 < kThreads, "a wave's maximum a thread");
    const int tid = threadIdx.x;
    float m = tid < a.nwave ? a.wavemax[static_cast<int64_t>(row) * a.nwave + tid] : -__builtin_inff();
    m = wave_max(m);
    if ((tid & 63) == 0) s.wave[tid >> 6] = __float_as_uint(m);
    __syncthreads();
    m = __uint_as_float(static_cast<uint32_t>(s.wave[tid & (kWaves - 1)]));
    m = row_max(m);  // 16 waves: every row of 16 lanes holds them all
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(m)));  // the same for every lane: a scalar
}

__device__ __forceinline__ Row row_of(const SampleArgs &a, int row, float t, float m) {
    Row r;
    r.l = row_buffer(a, row);
    r.n = a.n;
    r.nsub = a.nsub;
    r.m = m;
    r.m64 = static_cast<double>(m);
    r.infinite = m == __builtin_inff();
    r.rt = 1.0 / static_cast<double>(t);
    return r;
}

__device__ __forceinline__ void set_range(const Row &r, Ranges &g, int at, int first, int last) {
    g.first[at] = first;
    g.last[at] = last;
    g.lo[at] = first > last ? __builtin_inff() : last < kBins - 1 ? bin_floor(r, last) : -__builtin_inff();
    g.hi[at] = first > last ? -__builtin_inff() : bin_ceil(r, first);
}

// One workgroup per row and segment of it (segments first, so that a row spreads over
// the XCDs): the quick ways to their end (segment 0),
// or the segment's part of the row's histogram.
__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleArgs a) {
    __shared__ Shared s;
    const int row = blockIdx.y, tid = threadIdx.x, segment = blockIdx.x;
    Params p = params_of(a, row);
    if (p.quick() && !p.by_p && segment > 0) return;
    for (int i = tid; i < kBins; i += kThreads) {
        s.weight[i] = 0;
        s.count[i] = 0;
    }
    if (tid == 0) s.pick_at = 0xffffffffu;
    Subs subs;
    if (p.quick()) subs = load_subs(a, row);
    const float m = largest(s, a, row);
    const Row r = row_of(a, row, p.t, m);
    if (!(m > -__builtin_inff())) {  // no candidate
        if (segment == 0 && tid == 0) {
            write_row(a, row, -1, 0.f);
            a.state[row].phase = 1;
        }
        return;
    }
    bool whole = a.segments == 1;  // this workgroup makes the row's histogram alone
    int tail = kBins - 1;
    if (p.quick()) {
        if (p.greedy) {  // the lowest index among the largest
            for_tokens<1>(
                s, r, subs, [&](float sub) { return sub == m; }, [](const float *) { return true; },
                [&](int i, float l) { if (l == m) atomicMin(&s.pick_at, static_cast<uint32_t>(i)); });
            __syncthreads();
            if (tid == 0) {
                write_row(a, row, static_cast<int32_t>(s.pick_at), 1.f);
                a.state[row].phase = 1;
            }
            return;
        }
        int last = kBins - 1;
        if (p.by_k) {
            // the bin of the k-th largest maximum
#pragma unroll
            for (int q = 0; q < kSubsPerThread; ++q) {
                if (q * kThreads >= a.nsub) break;
                const int bin = bin_of(x_of(r, subs.v[q]));
                if (bin < kBins) atomicAdd(&s.count[bin], 1u);
            }
            if (tid == 0) s.pick_at = kBins - 1;
            __syncthreads();
            const int b0 = 2 * tid;
            const uint32_t c0 = s.count[b0], c1 = s.count[b0 + 1];
            u64 none = 0;
            uint32_t run = c0 + c1;
            block_scan(s, none, run);
            const uint32_t k = static_cast<uint32_t>(p.top_k);
            if (run >= k && run - c0 - c1 < k) s.pick_at = run - c1 >= k ? b0 : b0 + 1;
            __syncthreads();
            last = static_cast<int>(s.pick_at);
        } else if (p.min_p < 1.f) {
            // tokens with exp(-x) >= min_p, and a bin more for the rounding of the bound
            last = min(kBins - 1, static_cast<int>(fmin(bin_position(-log(static_cast<double>(p.min_p))), kBins - 1.0)) + 2);
        } else {
            last = 0;
        }
        Ranges g;
        set_range(r, g, 0, 0, last);
        set_range(r, g, 1, 0, -1);
        set_range(r, g, 2, 0, -1);
        bool many = false;
        if (p.by_p) {
            // min-p can keep any number of tokens.  Where half a thousand sub-blocks hold
            // one, all segments make the histogram (each decides this by itself).
            if (tid == 0) s.nsubs = 0;
            __syncthreads();
            uint32_t found = 0;
#pragma unroll
            for (int q = 0; q < kSubsPerThread; ++q) {
                if (q * kThreads >= a.nsub) break;
                found += static_cast<uint32_t>(__popcll(__ballot(subs.v[q] >= g.lo[0])));
            }
            if ((tid & 63) == 0 && found) atomicAdd(&s.nsubs, found);
            __syncthreads();
            many = s.nsubs > kQuick / 2;
            if (!many && segment > 0) return;
            tail = min(tail, last + 1);  // nothing behind is kept
        }
        if (!many) {
            const uint32_t near = gather(s, r, subs, g, 1, 0);
            if (near <= kQuick) {
                draw_from(s, a, r, p, row, g, Known{false, 0, 0}, static_cast<int>(near));
                if (tid == 0) a.state[row].phase = 1;
                return;
            }
            // too many tokens after all: this workgroup makes the whole row's histogram
            whole = true;
            if (tid == 0) a.state[row].phase = 2;
        }
        __syncthreads();
        for (int i = tid; i < kBins; i += kThreads) s.count[i] = 0;
        __syncthreads();
    }

    // Where only top-p ends the prefix, tokens with x over ln(n / (1 - top_p)) + 1 weigh
    // less than (1 - top_p) / e of the largest in all: the prefix ends before them.
    if (p.top_k == 0 && p.top_p < 1.f) {
        const double x = log(static_cast<double>(a.n) / (1.0 - static_cast<double>(fmaxf(p.top_p, 0.f)))) + 1.0;
        tail = static_cast<int>(fmin(bin_position(x) + 2.0, kBins - 1.0));
    }
    const int i0 = whole ? 0 : segment * a.segment, i1 = whole ? a.n : min(a.n, i0 + a.segment);
    u64 strong = add_tokens(s, r, p, i0, i1, tail);
    u64 *sums = a.sums + (static_cast<int64_t>(row) * a.segments + (whole ? 0 : segment)) * kSampleSums;
    uint32_t *counts = reinterpret_cast<uint32_t *>(sums + kBins);
    uint32_t none = 0;
    block_scan(s, strong, none);  // its barriers: the histogram is complete
    if (tid == kThreads - 1) sums[kSampleSums - 1] = strong;
    for (int i = tid; i < kBins; i += kThreads) {
        sums[i] = s.weight[i];
        if (p.top_k > 0) counts[i] = s.count[i];
    }
}

// Rows with a histogram: the ends of their prefixes.  Several workgroups a row gather
// the tokens that can hold an end; the last of them to finish (told by a counter)
// draws, from a list that it sorts: the order of arrival does not matter.
__global__ __launch_bounds__(kThreads) void sample_end_kernel(SampleArgs a) {
    __shared__ Shared s;
    const int row = blockIdx.y, tid = threadIdx.x;
    const uint32_t phase = a.state[row].phase;
    const int gathers = a.gathers, part = blockIdx.x;
    Params p = params_of(a, row);
    if (p.greedy) return;
    const int b0 = 2 * tid;
    // the sums of the segments' histograms; their loads need not wait for `phase`
    const u64 *sums = a.sums + static_cast<int64_t>(row) * a.segments * kSampleSums;
    u64 w0 = 0, w1 = 0, strong = 0;
    uint32_t c0 = 0, c1 = 0;
    const auto add = [&](int q) {
        const u64 *h = sums + static_cast<int64_t>(q) * kSampleSums;
        w0 += h[b0];
        w1 += h[b0 + 1];
        strong += h[kSampleSums - 1];
        if (p.top_k > 0) {
            const u64 c = h[kBins + tid];
            c0 += static_cast<uint32_t>(c);
            c1 += static_cast<uint32_t>(c >> 32);
        }
    };
    if (!p.quick()) {
#pragma unroll 8
        for (int q = 0; q < a.segments; ++q) add(q);
    }
    if (phase == 1) return;
    if (phase == 2) {  // only the first is there
        w0 = w1 = strong = 0;
        c0 = c1 = 0;
        add(0);
    } else if (p.quick()) {
        for (int q = 0; q < a.segments; ++q) add(q);
    }
    const Subs subs = load_subs(a, row);
    const float m = largest(s, a, row);
    const Row r = row_of(a, row, p.t, m);
    u64 run = w0 + w1;
    uint32_t run_c = c0 + c1;
    block_scan(s, run, run_c);
    s.weight[b0] = run - w1;
    s.weight[b0 + 1] = run;
    s.count[b0] = run_c - c1;
    s.count[b0 + 1] = run_c;
    __syncthreads();

    // the bin in which `cond` becomes true
    auto bin_with = [&](const EndTest &cond) {
        auto holds = [&](u64 w, uint32_t c) { return w > 0 && cond(w, c); };
        const bool before = holds(run - w1 - w0, run_c - c1 - c0), first = holds(run - w1, run_c - c1),
                   second = holds(run, run_c);
        if (!before && first) s.pick_at = b0;
        if (!first && second) s.pick_at = b0 + 1;
        __syncthreads();
        const int b = static_cast<int>(s.pick_at);
        __syncthreads();
        return b;
    };
    auto upto = [&](int b) { return b >= 0 ? s.weight[b] : 0; };
    const auto at_k = [&] { return EndTest{0, static_cast<uint32_t>(p.top_k), 0.0, 0}; };
    const auto at_p = [&](u64 sum) { return EndTest{1, 0, static_cast<double>(p.top_p) * static_cast<double>(sum), 0}; };
    const auto at_u = [&](u64 sum) { return EndTest{2, 0, static_cast<double>(p.u) * static_cast<double>(sum), sum}; };

    const u64 all = s.weight[kBins - 1];
    u64 kept = p.least > 0 ? strong : all;
    if (kept == 0) kept = static_cast<u64>(kUnit);  // min-p keeps one token at least
    const bool cut_k = p.top_k > 0 && static_cast<uint32_t>(p.top_k) < s.count[kBins - 1];
    if (!cut_k) p.top_k = 0;
    {
        // Every end's bin, or the few bins it can be in: C_k lies between its bin's
        // bounds, so the end of top-p between the ends for those, and the draw between
        // the draws for those.  All of these bins are gathered at once.
        const int bk = cut_k ? bin_with(at_k()) : -1;
        u64 low = cut_k ? upto(bk - 1) : all, high = cut_k ? upto(bk) : all;
        int p1 = -1, p2 = -2;
        if (p.top_p < 1.f) {
            p1 = p2 = bin_with(at_p(high));
            if (cut_k) p1 = bin_with(at_p(low));
            low = min(low, upto(p1 - 1));
            high = min(high, upto(p2));
        }
        low = min(low, kept);
        high = min(high, kept);
        const int d2 = bin_with(at_u(high)), d1 = low == high ? d2 : bin_with(at_u(low));
        Ranges g;
        set_range(r, g, 0, d1, d2);
        set_range(r, g, 1, p1, p2);
        set_range(r, g, 2, bk, cut_k ? bk : bk - 1);
        uint32_t near = gather(s, r, subs, g, gathers, part);
        if (gathers > 1) {
            // to the row's list in the workspace, as agent-scope stores (written through
            // to where the other XCDs read) that are complete before this workgroup counts
            RowState &st = a.state[row];
            u64 *list = a.near + static_cast<int64_t>(row) * kQuick;
            __syncthreads();
            if (tid == 0)
                s.fill = __hip_atomic_fetch_add(&st.fill, near, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            const uint32_t base = s.fill;
            if (static_cast<uint32_t>(tid) < near && base + tid < kQuick)
                __hip_atomic_store(list + base + tid, s.list[tid], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            __syncthreads();
            if (tid == 0)
                s.nsubs = __hip_atomic_fetch_add(&st.arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (s.nsubs != static_cast<uint32_t>(gathers) - 1) return;
            near = __hip_atomic_load(&st.fill, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (static_cast<uint32_t>(tid) < near)
                s.list[tid] = __hip_atomic_load(list + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
        }
        if (near <= kQuick) {
            draw_from(s, a, r, p, row, g, Known{true, all, kept}, static_cast<int>(near));
            return;
        }
        __syncthreads();
    }

    // More tokens than one a thread in those bins: one end after the other.
    u64 limit = all;
#pragma clang loop unroll(disable)
    for (int kind = 0; kind < 3; ++kind) {
        if (kind == 0 && !cut_k) continue;
        if (kind == 1 && !(p.top_p < 1.f)) continue;
        kept = min(kept, limit);
        const EndTest cond = kind == 0 ? at_k() : kind == 1 ? at_p(limit) : at_u(kept);
        const int b = bin_with(cond);
        Span sp;
        sp.bin = b;
        sp.klo = 0;
        sp.khi = 0xffffffffu;
        sp.llo = b < kBins - 1 ? bin_floor(r, b) : -__builtin_inff();
        sp.above = upto(b - 1);
        sp.above_c = b > 0 ? s.count[b - 1] : 0;
        if (cut_k) {
            sp.count = s.count[b] - sp.above_c;
        } else {
            // no counts are kept: a bound from the least weight a token of the bin has
            const double least = static_cast<double>(weight_of(x_at(b + 1.0))) * 0.999 - 1.0;
            const double most = least > 1.0 ? static_cast<double>(s.weight[b] - sp.above) / least + 1.0 : a.n;
            sp.count = most < a.n ? static_cast<uint32_t>(most) : static_cast<uint32_t>(a.n);
        }
        __syncthreads();
        const End e = find_end(s, r, subs, sp, cond);
        if (kind < 2)
            limit = e.sum;
        else if (tid == 0)
            write_draw(a, row, e.index, e.weight, kept);
    }
}

}  // namespace

hipError_t launch_sample(const SampleArgs &a, hipStream_t stream) {
    const int per = kMaxThreads * kMaxPerThread * 4;
    sample_max_kernel<<<dim3(a.rows, (a.n + per - 1) / per), kMaxThreads, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    sample_row_kernel<<<dim3(a.segments, a.rows), kThreads, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    sample_end_kernel<<<dim3(a.gathers, a.rows), kThreads, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace q8
