// moe_experts.hip -- the chosen experts' projections on vector instructions.
//
// Work split.  A wave streams a tile of 8 weight rows: lane 8 r + s takes row r
// and blocks s, s + 8, .., so that one step of the wave reads 272 contiguous bytes
// of each row, and the 8 lanes of a row meet at the end in three DPP adds (16 or 32
// lanes a row were no faster).  The activations are read through LDS, where the
// wave's 8 rows read the same addresses: staged once for the workgroup's eight
// waves (gate and up, which share them) or in pieces of each wave's own (down,
// whose waves have different experts).  One, two or four tokens a pass.
//
// Mathematics.  As in the GEMV: exact int32 block sums with v_dot4 (f64 products in
// the f32 mode), block terms (d s) T added in f64; g, u and h are rounded to f32 once
// each, as the projections' outputs are, and y once.
//
// Bound.  Reading the weights.  One token, two words: 8 experts of which 2 are chosen,
// k 4096, ff 14336 (375 MB): gate/up 47 us (5.3 TB/s), down 25 us (5.0 TB/s); with 64
// experts of which 8 are chosen, k 2048, ff 1408 (73 MB), 12 and 7.6 us, where the
// start of the launches counts.  Eight tokens of the latter: 50 and 37 us (5.1 and
// 3.4 TB/s).  The f32 mode is bound by its f64 products and conversions: 8 tokens of
// the same 84 and 64 us.
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
constexpr uint32_t kOob = 0x80000000u;  // an offset past every range: loads there read zeros

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// Bytes of a record: one block's words (f32 mode: its 32 values).
template <int WORDS>
constexpr int kRec = WORDS == 0 ? 128 : 32 * WORDS;
constexpr int kTokenGroup = 4;  // tokens one pass over a tile serves, at most
// Gate and up: two workgroups a CU.  In the f32 mode with four tokens a pass that cap on
// registers spills three of them (16 bytes a lane), and is faster all the same (81 against
// 92 us, below).  (Down: one, measured against two, which spilled more: 37 against 50 us.)
constexpr int kGateUpWaves = 4;  // of a SIMD

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, static_cast<int>(bytes), kBufferDword3);
}

// Activations of a launch: records [rows][nb] and block scales [rows][nb].
struct ActSource {
    __amdgpu_buffer_rsrc_t words, scales;
    int nb;
};

template <int WORDS>
__device__ __forceinline__ ActSource act_source(const void *words, const float *scales, int rows, int nb) {
    return ActSource{buffer_of(words, rows * nb * kRec<WORDS>), buffer_of(scales, WORDS ? rows * nb * 4 : 0), nb};
}

__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
    return make_uint4(v.x, v.y, v.z, v.w);
}
__device__ __forceinline__ float load_float(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}

// The weights of a wave: a tile of 8 rows of one expert's matrix, step by step.  Lane
// 8 r + s loads the window of block 8 step + s of row r; from `end` on (the row's last
// block, the wave's last step) it reads zeros and touches no memory.
struct Weights {
    __amdgpu_buffer_rsrc_t tile;
    uint32_t off;
    int step, end;

    __device__ __forceinline__ Weights(const uint8_t *w, int64_t first_row, int nb, int st0, int st1, int lane) {
        const uint32_t row_bytes = static_cast<uint32_t>(nb) * kBlockBytes;
        tile = buffer_of(w + first_row * row_bytes, kTileRows * row_bytes);
        step = st0;
        end = min(st1, (nb - (lane & 7) + kStepBlocks - 1) / kStepBlocks);
        off = (lane >> 3) * row_bytes + st0 * (kStepBlocks * kBlockBytes) + (((lane & 7) * kBlockBytes) & ~3u);
    }
    __device__ __forceinline__ void next(Window &w) {
        const uint32_t at = off | oob_bit(step < end);
        const u32x4 d0 = __builtin_amdgcn_raw_buffer_load_b128(tile, at, 0, 0);
        const u32x4 d1 = __builtin_amdgcn_raw_buffer_load_b128(tile, at + 16, 0, 0);
        w.d[8] = __builtin_amdgcn_raw_buffer_load_b32(tile, at + 32, 0, 0);
        w.d[0] = d0.x; w.d[1] = d0.y; w.d[2] = d0.z; w.d[3] = d0.w;
        w.d[4] = d1.x; w.d[5] = d1.y; w.d[6] = d1.z; w.d[7] = d1.w;
        off += kStepBlocks * kBlockBytes;
        ++step;
    }
};

// acc[t] += the block term of the lane's row and block with token t: the block's record
// is at rec + t * REC_STRIDE and its scale at sc[t * SC_STRIDE] (the 8 rows of a wave
// read the same addresses: broadcasts).
template <int WORDS, int TG, int REC_STRIDE, int SC_STRIDE>
__device__ __forceinline__ void compute(const Window &w, const uint8_t *rec, const float *sc, int lane, double (&acc)[TG]) {
    uint32_t q[8];
    window_quants(w, window_selector(lane & 7), q);
    const double d = static_cast<double>(f16_bits_to_float(window_scale_bits(w, lane & 7)));
#pragma unroll
    for (int t = 0; t < TG; ++t, rec += REC_STRIDE) {
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
            acc[t] += (d * static_cast<double>(sc[t * SC_STRIDE])) * static_cast<double>(tot);
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

template <int WORDS>
constexpr double kPost = WORDS == 2 ? 1.0 / 128.0 : 1.0;

// Hand LDS over between the waves of the workgroup; loads in flight stay in flight.
__device__ __forceinline__ void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    workgroup_barrier_acquire_lds();
}

// ------------------------------------------------------------------ gate and up

// Blocks of the tokens' rows that are in LDS at a time, for all waves.
template <int WORDS>
constexpr int kChunk = WORDS == 0 ? 64 : 128;

template <int WORDS, int MAX_TG>
struct GateUpShared {
    uint8_t words[MAX_TG][kChunk<WORDS> * kRec<WORDS>];
    float scales[MAX_TG][kChunk<WORDS>];
    float gu[MAX_TG][2][kHBlock];
};

// One pass: the wave's 8 rows of gate or up times n <= TG tokens, into s.gu.
template <int WORDS, int TG, typename S>
__device__ __forceinline__ void gate_up_pass(S &s, const uint8_t *w, int64_t first_row, const ActSource &src,
                                             const int *tokens, int n, int lane, int wave) {
    constexpr int C = kChunk<WORDS>, R = kRec<WORDS>;
    // windows in flight: 4 (3, 6 and 8 measured slower); in the f32 mode, whose conversions
    // need the registers, 2 (8 tokens, 64 experts of which 8 are chosen: 81 us; 4: 92, one
    // workgroup a CU and 4: 92)
    constexpr int kAhead = WORDS == 0 ? 2 : 4;
    static_assert(C * R <= kThreads * 16 && C * TG <= kThreads, "a load a thread and token, a scale a thread");
    const int tid = threadIdx.x;
    double acc[TG];
#pragma unroll
    for (int t = 0; t < TG; ++t) acc[t] = 0.0;
    for (int b0 = 0; b0 < src.nb; b0 += C) {
        const int nblk = min(C, src.nb - b0), steps = (nblk + kStepBlocks - 1) / kStepBlocks;
        // the first windows, which need nothing but the expert, then the tokens and the
        // chunk's activations (zeros behind the row's last block)
        Weights wt(w, first_row, src.nb, b0 / kStepBlocks, b0 / kStepBlocks + steps, lane);
        Window ring[kAhead];
#pragma unroll
        for (int p = 0; p < kAhead; ++p) wt.next(ring[p]);
        __builtin_amdgcn_sched_barrier(0);
        int rows[TG];
#pragma unroll
        for (int t = 0; t < TG; ++t) rows[t] = tokens ? tokens[min(t, n - 1)] : 0;
        uint4 v[TG];
#pragma unroll
        for (int t = 0; t < TG; ++t) {
            const bool ok = t < n && tid * 16 < nblk * R;
            v[t] = load16(src.words, ok ? (static_cast<uint32_t>(rows[t]) * src.nb + b0) * R + tid * 16 : kOob);
        }
        float sc = 0.f;
        if constexpr (WORDS > 0) {
            const int t = tid / C, i = tid % C;
            int row = rows[0];
#pragma unroll
            for (int u = 1; u < TG; ++u) row = t == u ? rows[u] : row;
            sc = load_float(src.scales, t < n && i < nblk ? (static_cast<uint32_t>(row) * src.nb + b0 + i) * 4 : kOob);
        }
        if (b0 > 0) lds_barrier();  // the last chunk has been read
#pragma unroll
        for (int t = 0; t < TG; ++t)
            if (tid * 16 < C * R) *reinterpret_cast<uint4 *>(s.words[t] + tid * 16) = v[t];
        if constexpr (WORDS > 0)
            if (tid < C * TG) s.scales[tid / C][tid % C] = sc;
        lds_barrier();
        const uint8_t *rec = s.words[0] + (lane & 7) * R;
        const float *scale = s.scales[0] + (lane & 7);
#pragma clang loop unroll(disable)
        for (int s0 = 0; s0 < steps; s0 += kAhead) {
#pragma unroll
            for (int p = 0; p < kAhead; ++p) {
                // a dead step's windows are zeros, and so is what the chunk holds behind its blocks.  (The
                // min changes no index; without it one token of large experts took 79.7 us, not 77.7.)
                static_assert(C / kStepBlocks % kAhead == 0, "dead steps stay in the chunk");
                const int at = min(s0 + p, C / kStepBlocks - 1);
                compute<WORDS, TG, C * R, C>(ring[p], rec + at * (kStepBlocks * R), scale + at * kStepBlocks, lane, acc);
                wt.next(ring[p]);
                __builtin_amdgcn_sched_barrier(0);  // one step's operands at a time in registers
            }
        }
    }
#pragma unroll
    for (int t = 0; t < TG; ++t) {
        const double tot = row_sum(acc[t]) * kPost<WORDS>;
        if (t < n && (lane & 7) == 0) s.gu[t][wave >> 2][(wave & 3) * kTileRows + (lane >> 3)] = static_cast<float>(tot);
    }
}

// One workgroup: one expert and 32 consecutive h values (the quantization block
// of the down projection's input).  Waves 0..3 take the gate rows, 4..7 the up
// rows; then a lane forms one h value, and the 32 lanes of a token quantize their
// block as quantize4 does, value for value.  MAX_TG: tokens a pass takes, at most;
// ONE: one token in the call.
template <int WORDS, int MAX_TG, bool ONE>
__global__ __launch_bounds__(kThreads, kGateUpWaves) void moe_gate_up_kernel(MoeArgs a) {
    __shared__ __align__(16) GateUpShared<WORDS, MAX_TG> s;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nhb = a.nbf;
    const int act = static_cast<int>(blockIdx.x) / nhb, hb = static_cast<int>(blockIdx.x) % nhb;
    // both loads at once (an entry behind the last is left over from another call)
    const MoeEntry en = a.plan->entry[act];
    const int n_active = a.plan->n_active;
    asm volatile("" ::"s"(en.expert), "s"(n_active));
    if (act >= n_active) return;
    const int count = ONE ? 1 : __popcll(en.mask);
    const uint8_t *w = wave < 4 ? a.w_gate : a.w_up;
    const int64_t first_row = static_cast<int64_t>(en.expert) * a.ff + hb * kHBlock + (wave & 3) * kTileRows;
    const ActSource src = act_source<WORDS>(WORDS ? static_cast<const void *>(a.xq) : a.x, a.xs, a.rows, a.nbk);
    for (int c0 = 0; c0 < count; c0 += MAX_TG) {
        const int n = min(MAX_TG, count - c0);
        const int *tokens = ONE ? nullptr : a.plan->pair_token + en.offset + c0;
        if (MAX_TG == 1 || n == 1)
            gate_up_pass<WORDS, 1>(s, w, first_row, src, tokens, n, lane, wave);
        else if (MAX_TG > 1 && n == 2)
            gate_up_pass<WORDS, MAX_TG == 1 ? 1 : 2>(s, w, first_row, src, tokens, n, lane, wave);
        else
            gate_up_pass<WORDS, MAX_TG>(s, w, first_row, src, tokens, n, lane, wave);
        __syncthreads();
        if (static_cast<int>(threadIdx.x) < n * kHBlock) {
            const int t = threadIdx.x / kHBlock, i = threadIdx.x % kHBlock;
            const double g = static_cast<double>(s.gu[t][0][i]), u = static_cast<double>(s.gu[t][1][i]);
            const float h = static_cast<float>(g / (1.0 + exp(-g)) * u);
            const int64_t blk = static_cast<int64_t>(en.offset + c0 + t) * a.nbf + hb;
            if constexpr (WORDS == 0) {
                reinterpret_cast<float *>(a.hq)[blk * kHBlock + i] = h;
            } else {
                float amax = fabsf(h);
#pragma unroll
                for (int off = 1; off < kHBlock; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
                const float sc = amax / 127.0f;
                const int q = sc == 0.0f ? 0 : quant_clamped(h / sc);
                int8_t *rec = reinterpret_cast<int8_t *>(a.hq) + blk * (WORDS * 32);
                rec[i] = static_cast<int8_t>(q);
                if constexpr (WORDS == 2) {
                    const float rest = __builtin_fmaf(-sc, static_cast<float>(q), h);
                    rec[32 + i] = static_cast<int8_t>(sc == 0.0f ? 0 : quant_clamped((rest * 128.0f) / sc));
                }
                if (i == 0) a.hs[blk] = sc;
            }
        }
        if (c0 + MAX_TG < count) __syncthreads();
    }
}

// ------------------------------------------------------------------------- down

// Steps of a pass whose activations a wave has in LDS at a time.
template <int TG>
constexpr int kSeg = TG == 4 ? 2 : 4;
template <int WORDS, int MAX_TG>
constexpr int kWaveBytes = MAX_TG * kSeg<MAX_TG> * kStepBlocks * kRec<WORDS>;

// One pass over steps [st0, st1) of the wave's tile for the tokens (pairs) first ..
// first + n - 1: f(token number, total of the lane's row).  The activations of kSeg
// steps at a time go through the wave's own piece of LDS, loaded a segment ahead as
// whole kilobytes: the loads of small pieces (one for each step and token) had cost
// more than the weights' at four tokens.
template <int WORDS, int TG, typename F>
__device__ __forceinline__ void down_pass(uint8_t *buf, float *sbuf, const uint8_t *w, int64_t first_row,
                                          const ActSource &src, int first, int n, int st0, int st1, int lane, F f) {
    constexpr int S = kSeg<TG>, R = kRec<WORDS>;
    constexpr int kSegBlocks = S * kStepBlocks, kSegBytes = kSegBlocks * R;
    constexpr int kLoads = (kSegBytes + 1023) / 1024;  // of 1 KB, per token and segment
    constexpr int kAhead = TG == 4 ? 2 : 4;            // windows in flight
    static_assert(TG * kSegBlocks <= 64, "a scale a lane");
    double acc[TG];
#pragma unroll
    for (int t = 0; t < TG; ++t) acc[t] = 0.0;
    uint4 v[TG][kLoads];
    float sc = 0.f;
    // zeros from st1 on: the ring's last steps have zero weights, and an infinite h there,
    // which is another wave's to add, would make the wave's sum NaN
    const int end = min(st1 * kStepBlocks, src.nb);
    auto load = [&](int st) {  // the segment that begins at step st
        const int b0 = st * kStepBlocks;
        const int nblk = min(kSegBlocks, end - b0);
#pragma unroll
        for (int t = 0; t < TG; ++t)
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int at = k * 1024 + lane * 16;
                const bool ok = t < n && at < nblk * R;
                v[t][k] = load16(src.words, ok ? (static_cast<uint32_t>(first + t) * src.nb + b0) * R + at : kOob);
            }
        if constexpr (WORDS > 0) {
            const int t = lane / kSegBlocks, i = lane % kSegBlocks;
            sc = load_float(src.scales, t < n && i < nblk ? (static_cast<uint32_t>(first + t) * src.nb + b0 + i) * 4 : kOob);
        }
    };
    load(st0);
    Weights wt(w, first_row, src.nb, st0, st1, lane);
    Window ring[kAhead];
#pragma unroll
    for (int p = 0; p < kAhead; ++p) wt.next(ring[p]);
    const uint8_t *rec = buf + (lane & 7) * R;
    const float *scale = sbuf + (lane & 7);
#pragma clang loop unroll(disable)
    for (int s0 = st0; s0 < st1; s0 += kAhead) {
#pragma unroll
        for (int p = 0; p < kAhead; ++p) {
            if (p % S == 0) {
                wave_lds_sync();  // the last segment has been read
#pragma unroll
                for (int t = 0; t < TG; ++t)
#pragma unroll
                    for (int k = 0; k < kLoads; ++k)
                        if (kSegBytes >= 1024 || lane * 16 < kSegBytes)
                            *reinterpret_cast<uint4 *>(buf + t * kSegBytes + k * 1024 + lane * 16) = v[t][k];
                if constexpr (WORDS > 0)
                    if (lane < TG * kSegBlocks) sbuf[lane] = sc;
                wave_lds_sync();
                load(s0 + p + S);
            }
            compute<WORDS, TG, kSegBytes, kSegBlocks>(ring[p], rec + (p % S) * (kStepBlocks * R), scale + (p % S) * kStepBlocks,
                                                      lane, acc);
            wt.next(ring[p]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int t = 0; t < TG; ++t)
        if (t < n) f(t, row_sum(acc[t]) * kPost<WORDS>);
}

// One workgroup: 8 output columns of y for every token.  The chosen experts'
// steps, laid end to end, are split evenly over the 8 waves; a wave adds
// gate * (its part of a product) to its own f64 sums [rows][8], and the waves'
// sums are added in wave order: the order of every sum depends on the choices
// alone.
template <int WORDS, int MAX_TG, bool ONE>
__global__ __launch_bounds__(kThreads, 2) void moe_down_kernel(MoeArgs a) {
    extern __shared__ __align__(16) double sums[];  // [waves][rows][8]
    __shared__ __align__(16) uint8_t bufs[kWaves][kWaveBytes<WORDS, MAX_TG>];
    __shared__ float sbufs[kWaves][64];
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
        const int count = ONE ? 1 : __popcll(en.mask);
        const int64_t first_row = static_cast<int64_t>(en.expert) * a.k + row0;
        for (int c0 = 0; c0 < count; c0 += MAX_TG) {
            const int first = en.offset + c0, n = min(MAX_TG, count - c0);
            const auto add = [&](int t, double tot) {
                const int token = ONE ? 0 : a.plan->pair_token[first + t];
                if ((lane & 7) == 0) mine[token * kTileRows + (lane >> 3)] += a.plan->pair_gate[first + t] * tot;
            };
            if (MAX_TG == 1 || n == 1)
                down_pass<WORDS, 1>(bufs[wave], sbufs[wave], a.w_down, first_row, src, first, n, st0, st1, lane, add);
            else if (MAX_TG > 1 && n == 2)
                down_pass<WORDS, MAX_TG == 1 ? 1 : 2>(bufs[wave], sbufs[wave], a.w_down, first_row, src, first, n, st0, st1, lane, add);
            else
                down_pass<WORDS, MAX_TG>(bufs[wave], sbufs[wave], a.w_down, first_row, src, first, n, st0, st1, lane, add);
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

template <int WORDS, int MAX_TG, bool ONE = false>
hipError_t run(const MoeArgs &a, hipStream_t stream) {
    // at most one expert per (token, choice)
    const int most = std::min(a.experts, a.rows * a.top_k);
    moe_gate_up_kernel<WORDS, MAX_TG, ONE><<<dim3(static_cast<unsigned>(most) * a.nbf), kThreads, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const size_t lds = static_cast<size_t>(kWaves) * a.rows * kTileRows * sizeof(double);
    moe_down_kernel<WORDS, MAX_TG, ONE><<<dim3(a.k / kTileRows), kThreads, lds, stream>>>(a);
    return hipGetLastError();
}

template <int WORDS>
hipError_t run_words(const MoeArgs &a, hipStream_t stream) {
    if (a.rows == 1) return run<WORDS, 1, true>(a, stream);
    return run<WORDS, kTokenGroup>(a, stream);
}

}  // namespace

hipError_t launch_moe_experts(int mode, const MoeArgs &a, hipStream_t stream) {
    if (a.tiled) return launch_moe_mma(mode, a, stream);
    return mode == 2 ? run_words<2>(a, stream) : mode == 1 ? run_words<1>(a, stream) : run_words<0>(a, stream);
}

}  // namespace q8
