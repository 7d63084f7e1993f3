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

// A tile of 8 rows of one expert's matrix, as a range-checked buffer.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t weight_tile(const uint8_t *w, int64_t first_row, int nb) {
    const uint32_t row_bytes = static_cast<uint32_t>(nb) * kBlockBytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t *>(w + first_row * row_bytes), 0,
                                             static_cast<int>(kTileRows * row_bytes), kBufferDword3);
}

template <int WORDS, int TG>
struct Step {
    Window w;
    uint32_t a[TG][kActDwords<WORDS>];
    float s[TG];
};

// Where a lane's loads of the next step are: its weight window (row lane / 8, block
// lane % 8 of the step), its piece of each token's words (block lane / 8), and its
// block's scales.  All move by a constant per step; from `w_end` and `a_end` on the
// lane's blocks are behind the row's last or behind the wave's steps, and the loads
// read zeros and touch no memory.
template <int WORDS, int TG>
struct Stream {
    __amdgpu_buffer_rsrc_t tile, words, scales;
    uint32_t w_off, a_off[TG], s_off[TG];
    int step, w_end, a_end;

    static constexpr int D = kActDwords<WORDS>;

    __device__ __forceinline__ Stream(__amdgpu_buffer_rsrc_t weights, const ActSource &src, const int (&arow)[TG], int st0,
                                      int st1, int lane) {
        tile = weights;
        words = src.words;
        scales = src.scales;
        step = st0;
        // the first step at which 8 step + (lane's block) >= nb
        w_end = min(st1, (src.nb - (lane & 7) + kStepBlocks - 1) / kStepBlocks);
        a_end = min(st1, (src.nb - (lane >> 3) + kStepBlocks - 1) / kStepBlocks);
        w_off = (lane >> 3) * static_cast<uint32_t>(src.nb) * kBlockBytes + st0 * (kStepBlocks * kBlockBytes) +
                (((lane & 7) * kBlockBytes) & ~3u);
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            const uint32_t block = static_cast<uint32_t>(arow[t]) * src.nb + st0 * kStepBlocks;
            const uint32_t dead = oob_bit(arow[t] >= 0);
            a_off[t] = ((block + (lane >> 3)) * (32 * D) + (lane & 7) * (4 * D)) | dead;
            s_off[t] = ((block + (lane & 7)) * 4) | dead;
        }
    }

    __device__ __forceinline__ void next(Step<WORDS, TG> &out) {
        const uint32_t w_dead = oob_bit(step < w_end), a_dead = oob_bit(step < a_end);
        const uint32_t off = w_off | w_dead;
        const u32x4 d0 = __builtin_amdgcn_raw_buffer_load_b128(tile, off, 0, 0);
        const u32x4 d1 = __builtin_amdgcn_raw_buffer_load_b128(tile, off + 16, 0, 0);
        out.w.d[8] = __builtin_amdgcn_raw_buffer_load_b32(tile, off + 32, 0, 0);
        out.w.d[0] = d0.x; out.w.d[1] = d0.y; out.w.d[2] = d0.z; out.w.d[3] = d0.w;
        out.w.d[4] = d1.x; out.w.d[5] = d1.y; out.w.d[6] = d1.z; out.w.d[7] = d1.w;
        w_off += kStepBlocks * kBlockBytes;
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            const uint32_t ao = a_off[t] | a_dead;
            if constexpr (D == 1) {
                out.a[t][0] = __builtin_amdgcn_raw_buffer_load_b32(words, ao, 0, 0);
            } else if constexpr (D == 2) {
                const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(words, ao, 0, 0);
                out.a[t][0] = v.x;
                out.a[t][1] = v.y;
            } else {
                const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(words, ao, 0, 0);
                out.a[t][0] = v.x; out.a[t][1] = v.y; out.a[t][2] = v.z; out.a[t][3] = v.w;
            }
            a_off[t] += kStepBlocks * 32 * D;
            if constexpr (WORDS > 0) {
                out.s[t] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(scales, s_off[t] | w_dead, 0, 0));
                s_off[t] += kStepBlocks * 4;
            }
        }
        ++step;
    }
};

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
__device__ __forceinline__ void run_steps(__amdgpu_buffer_rsrc_t wt, const ActSource &src, const int (&arow)[TG], int st0,
                                          int st1, uint8_t *buf, int lane, double (&acc)[TG]) {
    Stream<WORDS, TG> stream(wt, src, arow, st0, st1, lane);
    Step<WORDS, TG> ring[P];
#pragma unroll
    for (int p = 0; p < P; ++p) stream.next(ring[p]);
#pragma clang loop unroll(disable)
    for (int s0 = st0; s0 < st1; s0 += P) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            compute<WORDS, TG>(ring[p], buf, lane, acc);
            stream.next(ring[p]);
            __builtin_amdgcn_sched_barrier(0);  // one step's operands at a time in registers
        }
    }
}

constexpr int kTokenGroup = 4;  // tokens one pass over a tile serves, at most

// Steps in flight for a pass of TG tokens: as many loads ahead as registers allow at
// two workgroups a CU.
template <int TG>
constexpr int kAhead = TG == 4 ? 2 : TG == 2 ? 3 : 4;
// (one workgroup a CU in the f32 mode, whose conversions need the registers)
template <int WORDS>
constexpr int kWavesPerSimd = WORDS == 0 ? 2 : 4;

// One pass over steps [st0, st1) of a tile for tokens rows[0 .. n) (n at most
// kTokenGroup): f(token, total over the lanes of a row).
template <int WORDS, int TG, typename F>
__device__ __forceinline__ void pass_of(__amdgpu_buffer_rsrc_t wt, const ActSource &src, const int *rows, int n, int st0,
                                        int st1, uint8_t *buf, int lane, F f) {
    int arow[TG];
    double acc[TG];
#pragma unroll
    for (int t = 0; t < TG; ++t) {
        arow[t] = t < n ? rows[t] : -1;
        acc[t] = 0.0;
    }
    run_steps<WORDS, TG, kAhead<TG>>(wt, src, arow, st0, st1, buf, lane, acc);
#pragma unroll
    for (int t = 0; t < TG; ++t)
        if (t < n) f(t, row_sum(acc[t]) * (WORDS == 2 ? 1.0 / 128.0 : 1.0));
}

template <int WORDS, int MAX_TG, typename F>
__device__ __forceinline__ void pass(__amdgpu_buffer_rsrc_t wt, const ActSource &src, const int *rows, int n, int st0,
                                     int st1, uint8_t *buf, int lane, F f) {
    if (MAX_TG == 1 || n == 1)
        pass_of<WORDS, 1>(wt, src, rows, n, st0, st1, buf, lane, f);
    else if (MAX_TG > 1 && n == 2)
        pass_of<WORDS, 2>(wt, src, rows, n, st0, st1, buf, lane, f);
    else if (MAX_TG > 1)
        pass_of<WORDS, 4>(wt, src, rows, n, st0, st1, buf, lane, f);
}

template <int WORDS, int MAX_TG>
constexpr int kWaveBuf = MAX_TG * kStepBlocks * 32 * kActDwords<WORDS>;

// ------------------------------------------------------------------ gate and up

// One workgroup: one expert and 32 consecutive h values (the quantization block
// of the down projection's input).  Waves 0..3 take the gate rows, 4..7 the up
// rows; then a lane forms one h value, and the 32 lanes of a token quantize their
// block as quantize4 does, value for value.  MAX_TG = 1: one token in the call.
template <int WORDS, int MAX_TG>
__global__ __launch_bounds__(kThreads, kWavesPerSimd<WORDS>) void moe_gate_up_kernel(MoeArgs a) {
    __shared__ __align__(16) uint8_t bufs[kWaves][kWaveBuf<WORDS, MAX_TG>];
    __shared__ __align__(16) float gu[MAX_TG][2][kHBlock];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nhb = a.nbf;
    const int act = static_cast<int>(blockIdx.x) / nhb, hb = static_cast<int>(blockIdx.x) % nhb;
    if (act >= a.plan->n_active) return;
    const MoeEntry en = a.plan->entry[act];
    const int count = MAX_TG == 1 ? 1 : __popcll(en.mask);
    const uint8_t *w = wave < 4 ? a.w_gate : a.w_up;
    const __amdgpu_buffer_rsrc_t wt = weight_tile(w, static_cast<int64_t>(en.expert) * a.ff + hb * kHBlock + (wave & 3) * kTileRows,
                                                  a.nbk);
    const ActSource src = act_source<WORDS>(WORDS ? static_cast<const void *>(a.xq) : a.x, a.xs, a.rows, a.nbk);
    const int steps = (a.nbk + kStepBlocks - 1) / kStepBlocks;
    for (int c0 = 0; c0 < count; c0 += MAX_TG) {
        const int n = min(MAX_TG, count - c0);
        int rows[MAX_TG];
#pragma unroll
        for (int t = 0; t < MAX_TG; ++t)
            rows[t] = MAX_TG == 1 ? 0 : t < n ? a.plan->pair_token[en.offset + c0 + t] : -1;
        pass<WORDS, MAX_TG>(wt, src, rows, n, 0, steps, bufs[wave], lane, [&](int t, double tot) {
            if ((lane & 7) == 0) gu[t][wave >> 2][(wave & 3) * kTileRows + (lane >> 3)] = static_cast<float>(tot);
        });
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < n * kHBlock) {
            const int t = threadIdx.x / kHBlock, i = threadIdx.x % kHBlock;
            const double g = static_cast<double>(gu[t][0][i]), u = static_cast<double>(gu[t][1][i]);
            const float h = static_cast<float>(g / (1.0 + exp(-g)) * u);
            const int64_t blk = static_cast<int64_t>(en.offset + c0 + t) * a.nbf + hb;
            if constexpr (WORDS == 0) {
                reinterpret_cast<float *>(a.hq)[blk * kHBlock + i] = h;
            } else {
                float amax = fabsf(h);
#pragma unroll
                for (int off = 1; off < kHBlock; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
                const float s = amax / 127.0f;
                const int q = s == 0.0f ? 0 : quant_clamped(h / s);
                int8_t *rec = reinterpret_cast<int8_t *>(a.hq) + blk * (WORDS * 32);
                rec[i] = static_cast<int8_t>(q);
                if constexpr (WORDS == 2) {
                    const float rest = __builtin_fmaf(-s, static_cast<float>(q), h);
                    rec[32 + i] = static_cast<int8_t>(s == 0.0f ? 0 : quant_clamped((rest * 128.0f) / s));
                }
                if (i == 0) a.hs[blk] = s;
            }
        }
        if (c0 + MAX_TG < count) __syncthreads();
    }
}

// ------------------------------------------------------------------------- down

// One workgroup: 8 output columns of y for every token.  The chosen experts'
// steps, laid end to end, are split evenly over the 8 waves; a wave adds
// gate * (its part of a product) to its own f64 sums [rows][8], and the waves'
// sums are added in wave order: the order of every sum depends on the choices
// alone.
template <int WORDS, int MAX_TG>
__global__ __launch_bounds__(kThreads, kWavesPerSimd<WORDS>) void moe_down_kernel(MoeArgs a) {
    extern __shared__ __align__(16) double sums[];  // [waves][rows][8]
    __shared__ __align__(16) uint8_t bufs[kWaves][kWaveBuf<WORDS, MAX_TG>];
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
    for (int at = from; at < to;) {
        const int act = at / steps, st0 = at - act * steps;
        const int st1 = min(steps, st0 + to - at);
        at += st1 - st0;
        const MoeEntry en = a.plan->entry[act];
        const int count = MAX_TG == 1 ? 1 : __popcll(en.mask);
        const __amdgpu_buffer_rsrc_t wt = weight_tile(a.w_down, static_cast<int64_t>(en.expert) * a.k + row0, a.nbf);
        for (int c0 = 0; c0 < count; c0 += MAX_TG) {
            const int first = en.offset + c0;
            int rows[MAX_TG];
#pragma unroll
            for (int t = 0; t < MAX_TG; ++t) rows[t] = first + t;
            pass<WORDS, MAX_TG>(wt, src, rows, min(MAX_TG, count - c0), st0, st1, bufs[wave], lane, [&](int t, double tot) {
                const int token = MAX_TG == 1 ? 0 : a.plan->pair_token[first + t];
                if ((lane & 7) == 0) mine[token * kTileRows + (lane >> 3)] += a.plan->pair_gate[first + t] * tot;
            });
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

template <int WORDS, int MAX_TG>
hipError_t run(const MoeArgs &a, hipStream_t stream) {
    // at most one expert per (token, choice)
    const int most = std::min(a.experts, a.rows * a.top_k);
    moe_gate_up_kernel<WORDS, MAX_TG><<<dim3(static_cast<unsigned>(most) * a.nbf), kThreads, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const size_t lds = static_cast<size_t>(kWaves) * a.rows * kTileRows * sizeof(double);
    moe_down_kernel<WORDS, MAX_TG><<<dim3(a.k / kTileRows), kThreads, lds, stream>>>(a);
    return hipGetLastError();
}

template <int MAX_TG>
hipError_t run_mode(int mode, const MoeArgs &a, hipStream_t stream) {
    return mode == 2 ? run<2, MAX_TG>(a, stream) : mode == 1 ? run<1, MAX_TG>(a, stream) : run<0, MAX_TG>(a, stream);
}

}  // namespace

hipError_t launch_moe_experts(int mode, const MoeArgs &a, hipStream_t stream) {
    return a.rows == 1 ? run_mode<1>(mode, a, stream) : run_mode<kTokenGroup>(mode, a, stream);
}

}  // namespace q8
