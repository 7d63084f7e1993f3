// moe_experts.hip -- kernels and launchers described in moe_kernels.h.
#include <algorithm>

#include "moe_kernels.h"

#pragma clang fp contract(off)

namespace q8 {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kTileRows = 8;
constexpr int kStepBlocks = 8;
constexpr int kHBlock = 32;  // h values of one workgroup of the gate/up kernel: one quantization block
constexpr uint32_t kBufferDword3 = 0x00020000u;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Dwords of activation words a lane carries per token and step: the step's 8
// blocks of 32 values in 64 lanes.
template <int WORDS>
constexpr int kActDwords = WORDS == 0 ? 4 : WORDS;

// Activations of a launch: records of 32 values per block ([rows][nb] records
// of 4 * 8 * kActDwords bytes) and block scales [rows][nb].
struct ActSource {
    __amdgpu_buffer_rsrc_t words, scales;
    int nb;
};

template <int WORDS>
__device__ __forceinline__ ActSource act_source(const void *words, const float *scales, int rows, int nb) {
    ActSource s;
    s.words = __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(words), 0, rows * nb * (32 * kActDwords<WORDS>),
                                                kBufferDword3);
    s.scales = __builtin_amdgcn_make_buffer_rsrc(const_cast<float *>(scales), 0, WORDS ? rows * nb * 4 : 0,
                                                 kBufferDword3);
    s.nb = nb;
    return s;
}

// A tile of up to 8 rows of one expert's matrix, as a range-checked buffer.
struct WeightTile {
    __amdgpu_buffer_rsrc_t rsrc;
    uint32_t row_part;  // byte offset of the lane's row
};

__device__ __forceinline__ WeightTile weight_tile(const uint8_t *w, int64_t first_row, int nb, int lane) {
    WeightTile t;
    const uint32_t row_bytes = static_cast<uint32_t>(nb) * kBlockBytes;
    t.rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(w + first_row * row_bytes), 0,
                                               static_cast<int>(kTileRows * row_bytes), kBufferDword3);
    t.row_part = (lane >> 3) * row_bytes;
    return t;
}

template <int WORDS, int TG>
struct Step {
    Window w;
    uint32_t a[TG][kActDwords<WORDS>];
    float s[TG];
};

// Loads of step `st` (blocks 8 st .. 8 st + 7): nothing is read past nb blocks
// or for a token with base row -1 (zeros arrive instead).
template <int WORDS, int TG>
__device__ __forceinline__ void issue(const WeightTile &wt, const ActSource &src, const int (&arow)[TG], int st,
                                      bool live, int lane, Step<WORDS, TG> &out) {
    constexpr int D = kActDwords<WORDS>;
    const int b = st * kStepBlocks + (lane & 7);  // the lane's weight block
    const uint32_t off = (wt.row_part + (static_cast<uint32_t>(b * kBlockBytes) & ~3u)) | oob_bit(live && b < src.nb);
    const u32x4 d0 = __builtin_amdgcn_raw_buffer_load_b128(wt.rsrc, off, 0, 0);
    const u32x4 d1 = __builtin_amdgcn_raw_buffer_load_b128(wt.rsrc, off + 16, 0, 0);
    out.w.d[8] = __builtin_amdgcn_raw_buffer_load_b32(wt.rsrc, off + 32, 0, 0);
    out.w.d[0] = d0.x; out.w.d[1] = d0.y; out.w.d[2] = d0.z; out.w.d[3] = d0.w;
    out.w.d[4] = d1.x; out.w.d[5] = d1.y; out.w.d[6] = d1.z; out.w.d[7] = d1.w;
    const int ab = st * kStepBlocks + (lane >> 3);  // the block whose words the lane carries
#pragma unroll
    for (int t = 0; t < TG; ++t) {
        const bool ok = live && arow[t] >= 0;
        const uint32_t row = static_cast<uint32_t>(arow[t]) * src.nb;
        const uint32_t ao = ((row + ab) * (32 * D) + (lane & 7) * (4 * D)) | oob_bit(ok && ab < src.nb);
        if constexpr (D == 1) {
            out.a[t][0] = __builtin_amdgcn_raw_buffer_load_b32(src.words, ao, 0, 0);
        } else if constexpr (D == 2) {
            const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(src.words, ao, 0, 0);
            out.a[t][0] = v.x;
            out.a[t][1] = v.y;
        } else {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(src.words, ao, 0, 0);
            out.a[t][0] = v.x; out.a[t][1] = v.y; out.a[t][2] = v.z; out.a[t][3] = v.w;
        }
        if constexpr (WORDS > 0)
            out.s[t] = __uint_as_float(
                __builtin_amdgcn_raw_buffer_load_b32(src.scales, ((row + b) * 4) | oob_bit(ok && b < src.nb), 0, 0));
    }
}

// acc[t] += the step's block terms of the lane's row and block.
template <int WORDS, int TG>
__device__ __forceinline__ void compute(const Step<WORDS, TG> &st, uint8_t *buf, int lane, double (&acc)[TG]) {
    constexpr int D = kActDwords<WORDS>;
    constexpr int kRec = 32 * D;
    wave_lds_sync();  // the previous step's reads come first
#pragma unroll
    for (int t = 0; t < TG; ++t) {
        uint32_t *dst = reinterpret_cast<uint32_t *>(buf + t * kStepBlocks * kRec) + lane * D;
        if constexpr (D == 1)
            dst[0] = st.a[t][0];
        else if constexpr (D == 2)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(st.a[t][0], st.a[t][1]);
        else
            *reinterpret_cast<uint4 *>(dst) = make_uint4(st.a[t][0], st.a[t][1], st.a[t][2], st.a[t][3]);
    }
    wave_lds_sync();
    const int blk = lane & 7;
    uint32_t q[8];
    window_quants(st.w, window_selector(blk), q);
    const double d = static_cast<double>(f16_bits_to_float(window_scale_bits(st.w, blk)));
#pragma unroll
    for (int t = 0; t < TG; ++t) {
        const uint8_t *rec = buf + (t * kStepBlocks + blk) * kRec;
        if constexpr (WORDS == 0) {
            double p = 0.0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 xv = reinterpret_cast<const float4 *>(rec)[j];
                const uint32_t qw = q[j];
                p = __builtin_fma(static_cast<double>(static_cast<int8_t>(qw)), static_cast<double>(xv.x), p);
                p = __builtin_fma(static_cast<double>(static_cast<int8_t>(qw >> 8)), static_cast<double>(xv.y), p);
                p = __builtin_fma(static_cast<double>(static_cast<int8_t>(qw >> 16)), static_cast<double>(xv.z), p);
                p = __builtin_fma(static_cast<double>(static_cast<int8_t>(qw >> 24)), static_cast<double>(xv.w), p);
            }
            acc[t] += d * p;
        } else {
            uint32_t h[8], l[8];
            const uint4 h0 = reinterpret_cast<const uint4 *>(rec)[0], h1 = reinterpret_cast<const uint4 *>(rec)[1];
            h[0] = h0.x; h[1] = h0.y; h[2] = h0.z; h[3] = h0.w;
            h[4] = h1.x; h[5] = h1.y; h[6] = h1.z; h[7] = h1.w;
            int32_t tot = dot32(q, h);
            if constexpr (WORDS == 2) {
                const uint4 l0 = reinterpret_cast<const uint4 *>(rec)[2], l1 = reinterpret_cast<const uint4 *>(rec)[3];
                l[0] = l0.x; l[1] = l0.y; l[2] = l0.z; l[3] = l0.w;
                l[4] = l1.x; l[5] = l1.y; l[6] = l1.z; l[7] = l1.w;
                tot = tot * 128 + dot32(q, l);
            }
            acc[t] += (d * static_cast<double>(st.s[t])) * static_cast<double>(tot);
        }
    }
}

// Sum over the 8 lanes of a row; every one of them gets the total.
__device__ __forceinline__ double row_sum(double v) {
    v += dpp_f64<0xb1>(v);   // quad_perm [1,0,3,2]
    v += dpp_f64<0x4e>(v);   // quad_perm [2,3,0,1]
    v += dpp_f64<0x141>(v);  // row_half_mirror
    return v;
}

// Steps [st0, st1) of one tile and TG tokens, P steps in flight.
template <int WORDS, int TG, int P>
__device__ __forceinline__ void run_steps(const WeightTile &wt, const ActSource &src, const int (&arow)[TG], int st0,
                                          int st1, uint8_t *buf, int lane, double (&acc)[TG]) {
    Step<WORDS, TG> ring[P];
#pragma unroll
    for (int p = 0; p < P; ++p) issue<WORDS, TG>(wt, src, arow, st0 + p, st0 + p < st1, lane, ring[p]);
    for (int s0 = st0; s0 < st1; s0 += P) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            compute<WORDS, TG>(ring[p], buf, lane, acc);
            issue<WORDS, TG>(wt, src, arow, s0 + p + P, s0 + p + P < st1, lane, ring[p]);
        }
    }
}

constexpr int kTokenGroup = 4;  // tokens one pass over a tile serves

template <int WORDS>
constexpr int kWaveBuf = kTokenGroup * kStepBlocks * 32 * kActDwords<WORDS>;

// ------------------------------------------------------------------ gate and up

// One workgroup: one expert and 32 consecutive h values (the quantization block
// of the down projection's input).  Waves 0..3 take the gate rows, 4..7 the up
// rows.
template <int WORDS>
__global__ __launch_bounds__(kThreads) void moe_gate_up_kernel(MoeArgs a) {
    __shared__ __align__(16) uint8_t bufs[kWaves][kWaveBuf<WORDS>];
    __shared__ __align__(16) float gu[kTokenGroup][2][kHBlock];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nhb = a.nbf;
    const int act = static_cast<int>(blockIdx.x) / nhb, hb = static_cast<int>(blockIdx.x) % nhb;
    if (act >= a.plan->n_active) return;
    const MoeEntry en = a.plan->entry[act];
    const int count = __popcll(en.mask);
    const uint8_t *w = wave < 4 ? a.w_gate : a.w_up;
    const WeightTile wt = weight_tile(w, static_cast<int64_t>(en.expert) * a.ff + hb * kHBlock + (wave & 3) * kTileRows,
                                      a.nbk, lane);
    const ActSource src = act_source<WORDS>(WORDS ? static_cast<const void *>(a.xq) : a.x, a.xs, a.rows, a.nbk);
    const int steps = (a.nbk + kStepBlocks - 1) / kStepBlocks;
    const double post = WORDS == 2 ? 1.0 / 128.0 : 1.0;
    for (int c0 = 0; c0 < count; c0 += kTokenGroup) {
        int arow[kTokenGroup];
#pragma unroll
        for (int t = 0; t < kTokenGroup; ++t)
            arow[t] = c0 + t < count ? a.plan->pair_token[en.offset + c0 + t] : -1;
        double acc[kTokenGroup];
#pragma unroll
        for (int t = 0; t < kTokenGroup; ++t) acc[t] = 0.0;
        run_steps<WORDS, kTokenGroup, 2>(wt, src, arow, 0, steps, bufs[wave], lane, acc);
#pragma unroll
        for (int t = 0; t < kTokenGroup; ++t) {
            const double tot = row_sum(acc[t]) * post;
            if ((lane & 7) == 0) gu[t][wave >> 2][(wave & 3) * kTileRows + (lane >> 3)] = static_cast<float>(tot);
        }
        __syncthreads();
        if (threadIdx.x < kTokenGroup * kQuantLanes) {
            const int t = threadIdx.x / kQuantLanes, part = threadIdx.x % kQuantLanes;
            float h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const double g = static_cast<double>(gu[t][0][part * 4 + i]);
                const double u = static_cast<double>(gu[t][1][part * 4 + i]);
                h[i] = static_cast<float>(g / (1.0 + exp(-g)) * u);
            }
            const float4 hv = make_float4(h[0], h[1], h[2], h[3]);
            const int64_t blk = static_cast<int64_t>(en.offset + c0 + t) * a.nbf + hb;
            if constexpr (WORDS == 0) {
                if (c0 + t < count) reinterpret_cast<float4 *>(a.hq)[blk * kQuantLanes + part] = hv;
            } else {
                uint32_t h4, l4;
                const float s = quantize4<WORDS>(hv, h4, l4);
                if (c0 + t < count) {
                    uint32_t *rec = reinterpret_cast<uint32_t *>(a.hq + blk * (WORDS * 32));
                    rec[part] = h4;
                    if (WORDS == 2) rec[8 + part] = l4;
                    if (part == 0) a.hs[blk] = s;
                }
            }
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------- down

// One workgroup: 8 output columns of y for every token.  The chosen experts'
// steps, laid end to end, are split evenly over the 8 waves; a wave adds
// gate * (its part of a product) to its own f64 sums [rows][8], and the waves'
// sums are added in wave order: the order of every sum depends on the choices
// alone.
template <int WORDS>
__global__ __launch_bounds__(kThreads) void moe_down_kernel(MoeArgs a) {
    extern __shared__ __align__(16) double sums[];  // [waves][rows][8]
    __shared__ __align__(16) uint8_t bufs[kWaves][kWaveBuf<WORDS>];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int row0 = static_cast<int>(blockIdx.x) * kTileRows;
    double *mine = sums + wave * a.rows * kTileRows;
    for (int i = lane; i < a.rows * kTileRows; i += 64) mine[i] = 0.0;
    wave_lds_sync();
    const int steps = (a.nbf + kStepBlocks - 1) / kStepBlocks;
    const int n_active = a.plan->n_active;
    const int total = n_active * steps;
    const int from = static_cast<int>(static_cast<int64_t>(total) * wave / kWaves);
    const int to = static_cast<int>(static_cast<int64_t>(total) * (wave + 1) / kWaves);
    const ActSource src = act_source<WORDS>(a.hq, a.hs, a.rows * a.top_k, a.nbf);
    const double post = WORDS == 2 ? 1.0 / 128.0 : 1.0;
    for (int at = from; at < to;) {
        const int act = at / steps, st0 = at - act * steps;
        const int st1 = min(steps, st0 + to - at);
        at += st1 - st0;
        const MoeEntry en = a.plan->entry[act];
        const int count = __popcll(en.mask);
        const WeightTile wt = weight_tile(a.w_down, static_cast<int64_t>(en.expert) * a.k + row0, a.nbf, lane);
        for (int c0 = 0; c0 < count; c0 += kTokenGroup) {
            int arow[kTokenGroup];
            double acc[kTokenGroup];
#pragma unroll
            for (int t = 0; t < kTokenGroup; ++t) {
                arow[t] = c0 + t < count ? en.offset + c0 + t : -1;
                acc[t] = 0.0;
            }
            run_steps<WORDS, kTokenGroup, 2>(wt, src, arow, st0, st1, bufs[wave], lane, acc);
#pragma unroll
            for (int t = 0; t < kTokenGroup; ++t) {
                const double tot = row_sum(acc[t]) * post;
                if (c0 + t < count && (lane & 7) == 0) {
                    const int pair = en.offset + c0 + t;
                    mine[a.plan->pair_token[pair] * kTileRows + (lane >> 3)] += a.plan->pair_gate[pair] * tot;
                }
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.rows * kTileRows; i += kThreads) {
        double v = 0.0;
        for (int w = 0; w < kWaves; ++w) v += sums[w * a.rows * kTileRows + i];
        const int64_t o = static_cast<int64_t>(i / kTileRows) * a.k + row0 + i % kTileRows;
        if (a.residual) v += static_cast<double>(a.residual[o]);
        a.y[o] = static_cast<float>(v);
    }
}

template <int WORDS>
hipError_t run(const MoeArgs &a, hipStream_t stream) {
    // at most one expert per (token, choice)
    const int most = std::min(a.experts, a.rows * a.top_k);
    moe_gate_up_kernel<WORDS><<<dim3(static_cast<unsigned>(most) * a.nbf), kThreads, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const size_t lds = static_cast<size_t>(kWaves) * a.rows * kTileRows * sizeof(double);
    moe_down_kernel<WORDS><<<dim3(a.k / kTileRows), kThreads, lds, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_moe_experts(int mode, const MoeArgs &a, hipStream_t stream) {
    return mode == 2 ? run<2>(a, stream) : mode == 1 ? run<1>(a, stream) : run<0>(a, stream);
}

}  // namespace q8
