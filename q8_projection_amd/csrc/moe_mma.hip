// moe_mma.hip -- the chosen experts' projections on the matrix cores, for more than a
// few tokens an expert: int8 instructions in the integer modes, f64 in the f32 mode.
//
// Tiles.  v_mfma_i32_16x16x32_i8 takes one Q8_0 block of 16 weight rows against 16
// activation columns: lane l supplies bytes 8 q .. 8 q + 7 (q = l / 16) of row, or
// column, l % 16, and receives the exact sums of weight row l % 16 with columns
// 4 q .. 4 q + 3.  The columns are the tokens of one expert: 16 in the one-word mode,
// 8 (hi and lo words side by side) in the two-word mode.
//
// Weights go from memory to registers without LDS: lane (r, q) loads the window of
// block 4 s + q of row r, so that a step of the wave is 136 contiguous bytes of each
// of 16 rows, and a 4 x 4 exchange of 8-byte parts between the lanes of a row (eight
// swaps of half and quarter waves) turns four whole blocks in four lanes into four
// operands in every lane.  The activations are stored in the operands' order, and a
// lane reads its four parts as 32 contiguous bytes.
//
// The f32 mode multiplies scale times quant with the f32 values in
// v_mfma_f64_16x16x4f64: lane (r, q) supplies column j of block 4 s + q of its row for the
// j-th of 32 instructions a step, so that no exchange is needed, and receives weight row
// l % 16 with tokens q, q + 4, ...
//
// Sums.  Every block term (d s) T is added in f64, as everywhere in this library; g, u
// and h are rounded to f32 once each, as the projections' outputs are, and y once.
//
// Bound.  Reading the weights: 64 tokens, 64 experts of which 8 are chosen, k 2048, ff 1408
// (590 MB): gate/up 100 us (3.9 TB/s), down 69 us (2.8 TB/s), where the vector kernels read
// one token's large experts at 5.3 and 5.0.  The products are hidden behind the loads
// (without them each is 1 to 3 us faster); what is not is each workgroup's beginning and
// end: gate/up stages up to 66 KB of activations for 8 steps a wave and then joins and
// quantizes 32 values of h a token.
// The f32 mode is bound by its f64 instructions and the conversions beside them: 38
// tokens, 22 experts of which 8 are chosen, k 1408, ff 5184 (13.3 GFLOP, of which 16-token tiles
// make 17): gate/up 275 us, down 219 us.
#include <algorithm>
#include <type_traits>

#include "moe_kernels.h"

#pragma clang fp contract(off)

namespace q8 {
namespace {

constexpr int kTileRows = 16;
constexpr int kStepBlocks = 4;
constexpr int kHBlock = 32;  // h values of one workgroup of the gate/up kernel: one quantization block
constexpr uint32_t kBufferDword3 = 0x00020000u;
constexpr uint32_t kOob = 0x80000000u;  // an offset past every range: loads there read zeros

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef double v4d __attribute__((ext_vector_type(4)));

template <int WORDS>
struct Tile {
    static constexpr int kTokens = WORDS == 2 ? 8 : 16;  // tokens of a tile's 16 columns
    static constexpr int kVals = kTokens / 4;            // results a lane has of them
    static constexpr int kRec = WORDS == 0 ? 128 : WORDS * 32;  // bytes of a block of a token
    // column m: one word of one token; lane q's four columns are its kVals tokens' words
    static __device__ __forceinline__ int token(int m) { return WORDS == 2 ? m >> 1 : m; }
    static __device__ __forceinline__ int word(int m) { return WORDS == 2 ? m & 1 : 0; }
    // the token that lane q's result v is of, and the q and the v of a token
    static __device__ __forceinline__ int token_of(int q, int v) { return WORDS == 0 ? q + 4 * v : q * kVals + v; }
    static __device__ __forceinline__ int q_of(int token) { return WORDS == 0 ? token & 3 : token / kVals; }
    static __device__ __forceinline__ int v_of(int token) { return WORDS == 0 ? token >> 2 : token % kVals; }
};

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, static_cast<int>(bytes), kBufferDword3);
}

// 16 rows of one expert's matrix (k and ff are multiples of 64: whole tiles).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t weight_tile(const uint8_t *w, int64_t first_row, int nb) {
    const uint32_t row_bytes = static_cast<uint32_t>(nb) * kBlockBytes;
    return buffer_of(w + first_row * row_bytes, kTileRows * row_bytes);
}

// The window of the lane's block (row lane % 16, block 4 step + lane / 16); zeros for
// blocks behind the row's last and for steps that are not the wave's.
__device__ __forceinline__ void load_weights(__amdgpu_buffer_rsrc_t tile, uint32_t lane_off, int step, bool live,
                                             Window &w) {
    const uint32_t off = (lane_off + step * (kStepBlocks * kBlockBytes)) | oob_bit(live);
    const u32x4 d0 = __builtin_amdgcn_raw_buffer_load_b128(tile, off, 0, 0);
    const u32x4 d1 = __builtin_amdgcn_raw_buffer_load_b128(tile, off + 16, 0, 0);
    w.d[8] = __builtin_amdgcn_raw_buffer_load_b32(tile, off + 32, 0, 0);
    w.d[0] = d0.x; w.d[1] = d0.y; w.d[2] = d0.z; w.d[3] = d0.w;
    w.d[4] = d1.x; w.d[5] = d1.y; w.d[6] = d1.z; w.d[7] = d1.w;
}

// The activations of one token tile: the lane's operand parts of four blocks, and the
// block scales of its kVals tokens.
template <int WORDS>
struct Acts {
    long part[kStepBlocks];
    float s[Tile<WORDS>::kVals][kStepBlocks];
};

// f32 mode: the 32 values of the lane's token in the lane's block of the step.
template <>
struct Acts<0> {
    float4 x[8];
};

// Offsets of a lane's loads (of step 0), kOob where it has no token.
template <int WORDS>
struct ActOffsets {
    uint32_t part, s[Tile<WORDS>::kVals];
};

// `row(i)`: row of xq or hq of the tile's token i, or -1.
template <int WORDS, typename F>
__device__ __forceinline__ ActOffsets<WORDS> act_offsets(int sb, int lane, F row) {
    const int m = lane & 15, q = lane >> 4;
    ActOffsets<WORDS> o;
    const int mine = row(Tile<WORDS>::token(m));
    if constexpr (WORDS == 0) {
        o.part = mine >= 0 ? (static_cast<uint32_t>(mine) * sb + q) * 128 : kOob;
        return o;
    }
    o.part = mine >= 0 ? static_cast<uint32_t>(mine) * sb * (WORDS * 32) + Tile<WORDS>::word(m) * 128 + q * 32 : kOob;
#pragma unroll
    for (int v = 0; v < Tile<WORDS>::kVals; ++v) {
        const int r = row(q * Tile<WORDS>::kVals + v);
        o.s[v] = r >= 0 ? static_cast<uint32_t>(r) * sb * 4 : kOob;
    }
    return o;
}

template <int WORDS>
__device__ __forceinline__ void load_acts(__amdgpu_buffer_rsrc_t words, __amdgpu_buffer_rsrc_t scales,
                                          const ActOffsets<WORDS> &o, int step, bool live, Acts<WORDS> &a) {
    if constexpr (WORDS == 0) {
        const uint32_t off = (o.part + step * (kStepBlocks * 128)) | oob_bit(live);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(words, off + j * 16, 0, 0);
            a.x[j] = make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
        }
    } else {
        const uint32_t dead = oob_bit(live), off = (o.part + step * (WORDS * 128)) | dead;
        const u32x4 p0 = __builtin_amdgcn_raw_buffer_load_b128(words, off, 0, 0);
        const u32x4 p1 = __builtin_amdgcn_raw_buffer_load_b128(words, off + 16, 0, 0);
        a.part[0] = static_cast<long>((static_cast<uint64_t>(p0.y) << 32) | p0.x);
        a.part[1] = static_cast<long>((static_cast<uint64_t>(p0.w) << 32) | p0.z);
        a.part[2] = static_cast<long>((static_cast<uint64_t>(p1.y) << 32) | p1.x);
        a.part[3] = static_cast<long>((static_cast<uint64_t>(p1.w) << 32) | p1.z);
#pragma unroll
        for (int v = 0; v < Tile<WORDS>::kVals; ++v) {
            const u32x4 s = __builtin_amdgcn_raw_buffer_load_b128(scales, (o.s[v] + step * 16) | dead, 0, 0);
            a.s[v][0] = __uint_as_float(s.x); a.s[v][1] = __uint_as_float(s.y);
            a.s[v][2] = __uint_as_float(s.z); a.s[v][3] = __uint_as_float(s.w);
        }
    }
}

// (a, b) of lanes (q 0,1 | q 2,3): the upper half of a changes places with the lower half of b.
__device__ __forceinline__ void swap_halves(uint32_t &a, uint32_t &b) {
    const u32x2 r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r.x;
    b = r.y;
}
// The odd rows of 16 lanes of a change places with the even rows of b.
__device__ __forceinline__ void swap_rows(uint32_t &a, uint32_t &b) {
    const u32x2 r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r.x;
    b = r.y;
}

// The matrix-core operands and scales of four blocks of a lane's row.
struct Operands {
    long part[kStepBlocks];
    double d[kStepBlocks];
};

__device__ __forceinline__ void operands_of(const Window &w, int lane, Operands &o) {
    const int q = lane >> 4;  // the parity of the lane's block
    uint32_t e[8];
    window_quants(w, window_selector(q), e);
    // e[2p], e[2p + 1]: part p of block q.  Afterwards part q of block j is in e[2j], e[2j + 1].
    swap_halves(e[0], e[4]);
    swap_halves(e[1], e[5]);
    swap_halves(e[2], e[6]);
    swap_halves(e[3], e[7]);
    swap_rows(e[0], e[2]);
    swap_rows(e[1], e[3]);
    swap_rows(e[4], e[6]);
    swap_rows(e[5], e[7]);
#pragma unroll
    for (int j = 0; j < kStepBlocks; ++j)
        o.part[j] = static_cast<long>((static_cast<uint64_t>(e[2 * j + 1]) << 32) | e[2 * j]);
    // the four blocks' scales to all four lanes
    uint32_t d0 = __float_as_uint(f16_bits_to_float(window_scale_bits(w, q))), d2 = d0;
    swap_halves(d0, d2);
    uint32_t d1 = d0, d3 = d2;
    swap_rows(d0, d1);
    swap_rows(d2, d3);
    o.d[0] = static_cast<double>(__uint_as_float(d0));
    o.d[1] = static_cast<double>(__uint_as_float(d1));
    o.d[2] = static_cast<double>(__uint_as_float(d2));
    o.d[3] = static_cast<double>(__uint_as_float(d3));
}

// f32 mode: the lane's quants and scale.
struct RawOperands {
    uint32_t q[8];
    float d;
};
template <int WORDS>
using OperandsOf = std::conditional_t<WORDS == 0, RawOperands, Operands>;

__device__ __forceinline__ void operands_of(const Window &w, int lane, RawOperands &o) {
    window_quants(w, window_selector(lane >> 4), o.q);
    o.d = f16_bits_to_float(window_scale_bits(w, lane >> 4));
}

// f32 mode: acc[v] += the products of the lane's row with its tokens over the step's four
// blocks, one column of each block an instruction.  A scale (11 bits) times a quant (8) is
// exact in f32, and all that follows is f64.
__device__ __forceinline__ void multiply_f64(const RawOperands &w, const Acts<0> &a, double (&acc)[4]) {
    v4d sum = {acc[0], acc[1], acc[2], acc[3]};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float x[4] = {a.x[j].x, a.x[j].y, a.x[j].z, a.x[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float dw = w.d * static_cast<float>(static_cast<int8_t>(w.q[j] >> (8 * e)));
            sum = __builtin_amdgcn_mfma_f64_16x16x4f64(static_cast<double>(x[e]), static_cast<double>(dw), sum, 0, 0, 0);
        }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = sum[v];
}

// acc[v] += the four block terms of the lane's row with its tokens.
template <int WORDS>
__device__ __forceinline__ void multiply(const OperandsOf<WORDS> &w, const Acts<WORDS> &a, double (&acc)[Tile<WORDS>::kVals]) {
    if constexpr (WORDS == 0) {
        multiply_f64(w, a, acc);
        return;
    } else {
#pragma unroll
        for (int j = 0; j < kStepBlocks; ++j) {
            const v4i sum = __builtin_amdgcn_mfma_i32_16x16x32_i8(a.part[j], w.part[j], v4i{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < Tile<WORDS>::kVals; ++v) {
                const int t = WORDS == 2 ? sum[2 * v] * 128 + sum[2 * v + 1] : sum[v];
                acc[v] = __builtin_fma(w.d[j] * static_cast<double>(a.s[v][j]), static_cast<double>(t), acc[v]);
            }
        }
    }
}

// ------------------------------------------------------------------ gate and up

// Blocks of the tokens' rows that are in LDS at a time, for all waves, and the bytes
// between two rows there: 16 past a multiple of 128, so that the 16 columns' parts lie
// on different banks.
template <int WORDS>
constexpr int kChunk = WORDS == 0 ? 32 : 64;
template <int WORDS>
constexpr int kRowBytes = kChunk<WORDS> * Tile<WORDS>::kRec + 16;

constexpr int kParts = 2;                // waves that share the steps of a tile
constexpr int kGuWaves = 2 * kParts;     // small workgroups: two a CU, one's start and end beside the other's steps
constexpr int kGuThreads = 64 * kGuWaves;

template <int WORDS, int NT>
struct GateUpShared {
    static constexpr int kTokens = NT * Tile<WORDS>::kTokens;
    union {
        struct {
            uint8_t words[kTokens][kRowBytes<WORDS>];
            float scales[WORDS ? kTokens : 1][kChunk<WORDS>];
        };
        double part[kGuWaves][2][NT][Tile<WORDS>::kVals][64];
    };
};

// One workgroup: one expert and 32 consecutive h values (the quantization block of the
// down projection's input).  Eight waves and one workgroup a CU took 134 us where this
// takes 100, and more loads ahead (2, 3) or three workgroups of shorter chunks no less.  Wave w takes rows 16 (w / 2) .. of gate and of up, and
// every second step from w % 2 on; the two parts of a sum are added in order.  A pass takes
// up to NT token tiles; their rows are staged in LDS once for all waves, behind the
// first weight loads, so that the registers hold weights only.
template <int WORDS, int NT>
__global__ __launch_bounds__(kGuThreads, 2) void moe_gate_up_mma_kernel(MoeArgs a) {
    using T = Tile<WORDS>;
    using S = GateUpShared<WORDS, NT>;
    constexpr int kTokens = S::kTokens, C = kChunk<WORDS>, R = T::kRec, kAhead = 1;
    __shared__ __align__(16) S s;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int act = static_cast<int>(blockIdx.x) / a.nbf, hb = static_cast<int>(blockIdx.x) % a.nbf;
    // both loads at once (an entry behind the last is left over from another call)
    const MoeEntry en = a.plan->entry[act];
    const int n_active = a.plan->n_active;
    asm volatile("" ::"s"(en.expert), "s"(n_active));
    if (act >= n_active) return;
    const int count = __popcll(en.mask);
    const int64_t row0 = static_cast<int64_t>(en.expert) * a.ff + hb * kHBlock + (wave / kParts) * kTileRows;
    const __amdgpu_buffer_rsrc_t gate = weight_tile(a.w_gate, row0, a.nbk), up = weight_tile(a.w_up, row0, a.nbk);
    const __amdgpu_buffer_rsrc_t words = buffer_of(WORDS ? static_cast<const void *>(a.xq) : a.x, a.rows * a.sbk * R);
    const __amdgpu_buffer_rsrc_t scales = buffer_of(a.xs, WORDS ? a.rows * a.sbk * 4 : 0);
    const uint32_t lane_off = (lane & 15) * static_cast<uint32_t>(a.nbk) * kBlockBytes + (((lane >> 4) * kBlockBytes) & ~3u);
    const int w_end = (a.nbk - (lane >> 4) + kStepBlocks - 1) / kStepBlocks;  // steps in which the lane has a block
    const int m = lane & 15, q = lane >> 4;
    const int32_t *tokens = a.plan->pair_token + en.offset;
    for (int c0 = 0; c0 < count; c0 += kTokens) {
        const int n = min(kTokens, count - c0);
        double acc[2][NT][T::kVals];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int v = 0; v < T::kVals; ++v) acc[w][t][v] = 0.0;
        for (int b0 = 0; b0 < a.sbk; b0 += C) {
            const int nblk = min(C, a.sbk - b0), step0 = b0 / kStepBlocks, steps = (nblk + kStepBlocks - 1) / kStepBlocks;
            Window ring[kAhead][2];
            auto load = [&](int p, int w, int step) {
                load_weights(w ? up : gate, lane_off, step0 + step, step < steps && step0 + step < w_end, ring[p][w]);
            };
            const int first = wave % kParts;
#pragma unroll
            for (int p = 0; p < kAhead; ++p)
#pragma unroll
                for (int w = 0; w < 2; ++w) load(p, w, first + kParts * p);
            __builtin_amdgcn_sched_barrier(0);
            // 16 bytes a thread and load, every load in flight at once: the rows' words,
            // then their scales
            constexpr int kUnits = C * R / 16, kStep = kGuThreads / kUnits, kLoads = kTokens / kStep;
            constexpr int kScaleUnits = C / 4, kScaleStep = kGuThreads / kScaleUnits, kScaleLoads = (kTokens + kScaleStep - 1) / kScaleStep;
            static_assert(kGuThreads % kUnits == 0 && kTokens % kStep == 0, "whole rows");
            const int unit = tid % kUnits, scale_unit = tid % kScaleUnits;
            uint32_t row[kLoads], scale_row[kScaleLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) row[k] = static_cast<uint32_t>(tokens[c0 + min(tid / kUnits + k * kStep, n - 1)]);
#pragma unroll
            for (int k = 0; k < kScaleLoads; ++k)
                scale_row[k] = static_cast<uint32_t>(tokens[c0 + min(tid / kScaleUnits + k * kScaleStep, n - 1)]);
            u32x4 d[kLoads], ds[kScaleLoads];
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const bool ok = k * kStep < n && unit * 16 < nblk * R;
                d[k] = __builtin_amdgcn_raw_buffer_load_b128(words, ok ? (row[k] * a.sbk + b0) * R + unit * 16 : kOob, 0, 0);
            }
#pragma unroll
            for (int k = 0; WORDS && k < kScaleLoads; ++k)
                ds[k] = __builtin_amdgcn_raw_buffer_load_b128(
                    scales, scale_unit * 4 < nblk ? (scale_row[k] * a.sbk + b0 + scale_unit * 4) * 4 : kOob, 0, 0);
            if (c0 > 0 || b0 > 0) __syncthreads();  // what was there has been read
#pragma unroll
            for (int k = 0; k < kLoads; ++k)
                *reinterpret_cast<u32x4 *>(s.words[tid / kUnits + k * kStep] + unit * 16) = d[k];
#pragma unroll
            for (int k = 0; WORDS && k < kScaleLoads; ++k)
                if (tid / kScaleUnits + k * kScaleStep < kTokens)
                    *reinterpret_cast<u32x4 *>(&s.scales[tid / kScaleUnits + k * kScaleStep][scale_unit * 4]) = ds[k];
            __syncthreads();
#pragma clang loop unroll(disable)
            for (int s0 = first; s0 < steps; s0 += kParts * kAhead) {
#pragma unroll
                for (int p = 0; p < kAhead; ++p) {
                    const int st = min(s0 + kParts * p, steps - 1);  // (a step behind the last has zero weights)
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        OperandsOf<WORDS> o;
                        operands_of(ring[p][w], lane, o);
                        load(p, w, s0 + kParts * (p + kAhead));
#pragma unroll
                        for (int t = 0; t < NT; ++t) {
                            if (t * T::kTokens >= n) break;  // the same for the workgroup
                            Acts<WORDS> x;
                            // columns without a token repeat the last one: their sums are not used
                            const uint8_t *row = s.words[min(t * T::kTokens + T::token(m), n - 1)] + st * (kStepBlocks * R);
                            if constexpr (WORDS == 0) {
#pragma unroll
                                for (int j = 0; j < 8; ++j) x.x[j] = reinterpret_cast<const float4 *>(row + q * 128)[j];
                            } else {
                                const ulonglong2 *part = reinterpret_cast<const ulonglong2 *>(row + T::word(m) * 128 + q * 32);
                                const ulonglong2 p0 = part[0], p1 = part[1];
                                x.part[0] = static_cast<long>(p0.x); x.part[1] = static_cast<long>(p0.y);
                                x.part[2] = static_cast<long>(p1.x); x.part[3] = static_cast<long>(p1.y);
#pragma unroll
                                for (int v = 0; v < T::kVals; ++v) {
                                    const float4 sv = *reinterpret_cast<const float4 *>(
                                        &s.scales[min(t * T::kTokens + q * T::kVals + v, n - 1)][st * 4]);
                                    x.s[v][0] = sv.x; x.s[v][1] = sv.y; x.s[v][2] = sv.z; x.s[v][3] = sv.w;
                                }
                            }
                            multiply<WORDS>(o, x, acc[w][t]);
                            __builtin_amdgcn_sched_barrier(0);  // one tile's operands at a time in registers
                        }
                    }
                }
            }
        }
        __syncthreads();  // the activations have been read
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int v = 0; v < T::kVals; ++v) s.part[wave][w][t][v][lane] = acc[w][t][v];
        __syncthreads();
        // a thread forms one h value; the 32 of a token quantize their block as quantize4 does
        for (int i = threadIdx.x; i < n * kHBlock; i += kGuThreads) {
            const int token = i / kHBlock, row = i % kHBlock;
            const int t = token / T::kTokens, in = token % T::kTokens;
            const int from = T::q_of(in) * 16 + (row & 15), v = T::v_of(in);
            double sums[2];
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                const int w0 = (row >> 4) * kParts;
                sums[m] = s.part[w0][m][t][v][from];
#pragma unroll
                for (int w = 1; w < kParts; ++w) sums[m] += s.part[w0 + w][m][t][v][from];
            }
            const double post = WORDS == 2 ? 1.0 / 128.0 : 1.0;
            const double g = static_cast<double>(static_cast<float>(sums[0] * post));
            const double u = static_cast<double>(static_cast<float>(sums[1] * post));
            const float h = static_cast<float>(g / (1.0 + exp(-g)) * u);
            const int64_t pair = en.offset + c0 + token;
            if constexpr (WORDS == 0) {
                reinterpret_cast<float *>(a.hq)[(pair * a.nbf + hb) * kHBlock + row] = h;
            } else {
                float amax = fabsf(h);
#pragma unroll
                for (int off = 1; off < kHBlock; off <<= 1) amax = fmaxf(amax, __shfl_xor(amax, off, 64));
                const float sc = amax / 127.0f;
                const int hi = sc == 0.0f ? 0 : quant_clamped(h / sc);
                uint8_t *rec = a.hq + pair * a.sbf * (WORDS * 32);
                rec[record_offset(1, WORDS, hb, 0, row >> 2) + (row & 3)] = static_cast<uint8_t>(hi);
                if constexpr (WORDS == 2) {
                    const float rest = __builtin_fmaf(-sc, static_cast<float>(hi), h);
                    const int l = sc == 0.0f ? 0 : quant_clamped((rest * 128.0f) / sc);
                    rec[record_offset(1, WORDS, hb, 1, row >> 2) + (row & 3)] = static_cast<uint8_t>(l);
                }
                if (row == 0) a.hs[pair * a.sbf + hb] = sc;
                // the blocks that round the row up to four have scale 0 (their words meet zero weights)
                if (hb == a.nbf - 1 && row < a.sbf - a.nbf) a.hs[pair * a.sbf + a.nbf + row] = 0.f;
            }
        }
    }
}

// ------------------------------------------------------------------------- down

// A tile of 32 output columns of y for every token, by a.splits workgroups.  The chosen
// experts' steps, laid end to end, are split evenly over the workgroups' waves; a wave
// adds gate * (its part of a product) to its own f64 sums [rows][32], the waves' sums
// are added in wave order, and the workgroups' sums (through the workspace, by the last
// to arrive) in their order: the order of every sum depends on the choices alone.  Two
// tiles of 16 columns a wave share the activations' loads (16 columns and eight waves: 87
// us, these: 74); two steps ahead, or the loads of the next expert during the last steps
// of one, were worth 2 us of 74 and are not here.
constexpr int kDownWaves = 4, kDownThreads = 64 * kDownWaves;
static_assert(kMoeDownRows == 2 * kTileRows, "two tiles a wave");

template <int WORDS, int NT>
__global__ __launch_bounds__(kDownThreads, 2) void moe_down_mma_kernel(MoeArgs a) {
    using T = Tile<WORDS>;
    constexpr int kTokens = NT * T::kTokens;
    constexpr int kAhead = 1;
    extern __shared__ __align__(16) double sums[];  // [waves][rows][32]
    __shared__ int is_last;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // workgroups in turn take different tiles of the same part: every XCD then has a share of
    // each expert (72 us where an XCD had experts of its own, 69 so)
    const int tiles = a.k / kMoeDownRows;
    const int tile = static_cast<int>(blockIdx.x) % tiles, split = static_cast<int>(blockIdx.x) / tiles;
    const int row0 = tile * kMoeDownRows;
    const int outs = a.rows * kMoeDownRows;
    double *mine = sums + wave * outs;
    for (int i = lane; i < outs; i += 64) mine[i] = 0.0;
    wave_lds_sync();
    const int steps = (a.sbf + kStepBlocks - 1) / kStepBlocks;
    const int total = a.plan->n_active * steps;
    const int me = split * kDownWaves + wave, all = a.splits * kDownWaves;
    const int from = static_cast<int>(static_cast<int64_t>(total) * me / all);
    const int to = static_cast<int>(static_cast<int64_t>(total) * (me + 1) / all);
    const __amdgpu_buffer_rsrc_t words = buffer_of(a.hq, a.rows * a.top_k * a.sbf * T::kRec);
    const __amdgpu_buffer_rsrc_t scales = buffer_of(a.hs, WORDS ? a.rows * a.top_k * a.sbf * 4 : 0);
    const uint32_t lane_off = (lane & 15) * static_cast<uint32_t>(a.nbf) * kBlockBytes + (((lane >> 4) * kBlockBytes) & ~3u);
    const int w_end = (a.nbf - (lane >> 4) + kStepBlocks - 1) / kStepBlocks;
    const double post = WORDS == 2 ? 1.0 / 128.0 : 1.0;
    for (int at = from; at < to;) {
        const int act = at / steps, st0 = at - act * steps;
        const int st1 = min(steps, st0 + to - at);
        at += st1 - st0;
        const MoeEntry en = a.plan->entry[act];
        const int count = __popcll(en.mask);
        const int64_t row = static_cast<int64_t>(en.expert) * a.k + row0;
        const __amdgpu_buffer_rsrc_t wt[2] = {weight_tile(a.w_down, row, a.nbf), weight_tile(a.w_down, row + kTileRows, a.nbf)};
        for (int c0 = 0; c0 < count; c0 += kTokens) {
            ActOffsets<WORDS> ao[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t)
                ao[t] = act_offsets<WORDS>(a.sbf, lane, [&](int i) {
                    const int p = c0 + t * T::kTokens + i;
                    return p < count ? en.offset + p : -1;
                });
            double acc[2][NT][T::kVals];
#pragma unroll
            for (int w = 0; w < 2; ++w)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int v = 0; v < T::kVals; ++v) acc[w][t][v] = 0.0;
            struct {
                Window w[2];
                Acts<WORDS> acts[NT];
            } ring[kAhead];
            auto load = [&](int p, int step) {
#pragma unroll
                for (int w = 0; w < 2; ++w) load_weights(wt[w], lane_off, step, step < min(st1, w_end), ring[p].w[w]);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (c0 + t * T::kTokens < count) load_acts<WORDS>(words, scales, ao[t], step, step < (WORDS ? st1 : min(st1, w_end)), ring[p].acts[t]);
            };
#pragma unroll
            for (int p = 0; p < kAhead; ++p) load(p, st0 + p);
#pragma clang loop unroll(disable)
            for (int s0 = st0; s0 < st1; s0 += kAhead) {
#pragma unroll
                for (int p = 0; p < kAhead; ++p) {
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        OperandsOf<WORDS> o;
                        operands_of(ring[p].w[w], lane, o);
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            if (c0 + t * T::kTokens < count) multiply<WORDS>(o, ring[p].acts[t], acc[w][t]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    load(p, s0 + p + kAhead);
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int v = 0; v < T::kVals; ++v) {
                    const int p = c0 + t * T::kTokens + T::token_of(lane >> 4, v);
                    if (p >= count) continue;
                    double *out = mine + a.plan->pair_token[en.offset + p] * kMoeDownRows + (lane & 15);
                    const double gate = a.plan->pair_gate[en.offset + p];
                    out[0] += gate * (acc[0][t][v] * post);
                    out[kTileRows] += gate * (acc[1][t][v] * post);
                }
        }
    }
    __syncthreads();
    double *parts = a.parts + static_cast<int64_t>(tile) * a.splits * outs;
    if (a.splits > 1) {
        // agent-scope stores, complete before this workgroup counts itself in
        for (int i = threadIdx.x; i < outs; i += kDownThreads) {
            double v = 0.0;
            for (int w = 0; w < kDownWaves; ++w) v += sums[w * outs + i];
            __hip_atomic_store(parts + static_cast<int64_t>(split) * outs + i, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (threadIdx.x == 0) {
            uint32_t *counter = a.counters + kMoeTileCounter + tile;
            const uint32_t done = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            is_last = done == static_cast<uint32_t>(a.splits) - 1;
            if (is_last) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
        __syncthreads();
        if (!is_last) return;
    }
#pragma unroll 2
    for (int i = threadIdx.x; i < outs; i += kDownThreads) {
        double v = 0.0;
        if (a.splits > 1) {
            double part[kMoeMaxSplits];  // every load in flight at once
#pragma unroll
            for (int s = 0; s < kMoeMaxSplits; ++s)
                part[s] = s < a.splits ? __hip_atomic_load(parts + static_cast<int64_t>(s) * outs + i, __ATOMIC_RELAXED,
                                                           __HIP_MEMORY_SCOPE_AGENT) : 0.0;
#pragma unroll
            for (int s = 0; s < kMoeMaxSplits; ++s) v += part[s];
        } else {
            for (int w = 0; w < kDownWaves; ++w) v += sums[w * outs + i];
        }
        const int64_t o = static_cast<int64_t>(i / kMoeDownRows) * a.k + row0 + i % kMoeDownRows;
        if (a.residual) v += static_cast<double>(a.residual[o]);
        a.y[o] = static_cast<float>(v);
    }
}

template <int WORDS, int NT>
hipError_t run(const MoeArgs &a, hipStream_t stream) {
    const int most = std::min(a.experts, a.rows * a.top_k);
    moe_gate_up_mma_kernel<WORDS, NT><<<dim3(static_cast<unsigned>(most) * a.nbf), kGuThreads, 0, stream>>>(a);
    if (hipError_t e = hipGetLastError(); e != hipSuccess) return e;
    const size_t lds = static_cast<size_t>(kDownWaves) * a.rows * kMoeDownRows * sizeof(double);
    moe_down_mma_kernel<WORDS, NT><<<dim3(a.k / kMoeDownRows * a.splits), kDownThreads, lds, stream>>>(a);
    return hipGetLastError();
}

template <int WORDS>
hipError_t run_words(const MoeArgs &a, hipStream_t stream) {
    // token tiles a pass, by the mean number of tokens an expert gets.  One tile and two, in
    // us a layer (64 experts of which 8 are chosen, k 2048, ff 1408), two words, 8 tokens a
    // tile: mean 3: 150, 155; 4: 163, 158; 5: 184, 166; 8: 220, 182.  One word, 16 tokens:
    // mean 4: 160, 160; 8: 177, 177; 16 (32 experts): 134, 115.  f32 mode: one (gate/up at a
    // mean of 8: 241, 265; the activations of two do not fit the registers of down).
    if constexpr (WORDS == 0) {
        return run<WORDS, 1>(a, stream);
    } else {
        const int mean = a.rows * a.top_k / a.experts;
        return 2 * mean >= Tile<WORDS>::kTokens ? run<WORDS, 2>(a, stream) : run<WORDS, 1>(a, stream);
    }
}

}  // namespace

hipError_t launch_moe_mma(int mode, const MoeArgs &a, hipStream_t stream) {
    return mode == 2 ? run_words<2>(a, stream) : mode == 1 ? run_words<1>(a, stream) : run_words<0>(a, stream);
}

}  // namespace q8
