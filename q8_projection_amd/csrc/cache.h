// cache.h -- the key/value cache's layout (q8_cache.h) and what its kernels and
// the attention's take.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q8 {

constexpr int kTileTokens = 32;

struct CacheArgs {
    uint8_t *data;
    int64_t pages;
    int kv_heads;
    int page_shift;        // log2 of a page's tokens
    int sequences;
    int64_t table_ld;
    const int32_t *table;  // [sequences][table_ld]
    const int32_t *lens;   // [sequences]
    const int32_t *starts; // [sequences + 1] or null: row s is sequence s's
    int rows;
    int max_rows;          // of one sequence, at most `rows`
};

struct AppendArgs {
    CacheArgs c;
    const float *k, *v;
    int64_t k_ld, v_ld;
};

struct ReadArgs {
    CacheArgs c;
    float *k, *v;  // [rows][kv_heads][D]
};

struct AttentionArgs {
    CacheArgs c;
    const float *q;
    int64_t q_ld;
    int heads;
    int group;     // query heads of a kv head
    float scale;
    int window;    // 0: no window
    float *out;
    float *lse;    // or null
};

// A tile's parts, in bytes from its start.
template <int BITS, int D>
struct Tile {
    static constexpr int kBlocks = D / 32;
    static constexpr int kRow = D * BITS / 8;             // key codes of one token
    static constexpr int kKeyWords = kTileTokens * kRow;
    static constexpr int kWords = kTileTokens * kBlocks * 2;
    static constexpr int kValues = kKeyWords + kWords;
    static constexpr int kValueWords = kValues + kTileTokens * kRow;
    static constexpr int kBytes = kValueWords + kWords;
};

inline int64_t tile_bytes(int bits, int d) { return int64_t(2) * kTileTokens * (d * bits / 8 + d / 32 * 2); }

// Places of a token's words in their part: [a][b][block][i] and [block][a][b][i], as 16-bit words.
__device__ __forceinline__ int key_word(int t, int block, int blocks) {
    return (((t >> 3) * 4 + (t & 3)) * blocks + block) * 2 + ((t >> 2) & 1);
}
__device__ __forceinline__ int value_word(int t, int block) {
    return (block * 4 + (t >> 3)) * 8 + (t & 3) * 2 + ((t >> 2) & 1);
}

__device__ __forceinline__ float half_value(uint32_t bits) {
    return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits)));
}

// The value of a code under its block's word.
template <int BITS>
__device__ __forceinline__ float value_of(uint32_t word, uint32_t code) {
    if (BITS == 4) return half_value(word & 0x7fe0u) * static_cast<float>(static_cast<int>(code) - static_cast<int>(word & 15u));
    return half_value(word) * static_cast<float>(static_cast<int>(code) - 128);
}

// A sequence of a call: its rows, clipped to the call's arrays, and where they are.
struct Rows {
    int first;     // its first row
    int n;         // rows that the call serves
    int at;        // token of the first row (negative: no token)
    int end;       // tokens that the cache can hold of it: lens within 0 .. capacity
};

__device__ __forceinline__ Rows sequence_rows(const CacheArgs &c, int s) {
    Rows r;
    const int len = min(max(c.lens[s], 0), 1 << 30);
    int64_t first = s, n = 1;
    if (c.starts) {
        first = c.starts[s];
        n = c.starts[s + 1] - first;
        if (first < 0 || first > c.rows) first = n = 0;
        n = n < 0 ? 0 : n;
        n = n > c.rows - first ? c.rows - first : n;
    }
    r.first = static_cast<int>(first);
    r.at = len - static_cast<int>(n);
    r.n = static_cast<int>(n) < c.max_rows ? static_cast<int>(n) : c.max_rows;
    const int64_t capacity = c.table_ld << c.page_shift;  // at most 2^30
    r.end = len < capacity ? len : static_cast<int>(capacity);
    return r;
}

// The tile of tokens 32 t .. of sequence s and a kv head, or null if no page of the pool holds it.
template <int BITS, int D>
__device__ __forceinline__ uint8_t *tile_at(const CacheArgs &c, int s, int t, int head) {
    const int shift = c.page_shift - 5;  // a page's tiles
    const int64_t page = c.table[s * c.table_ld + (t >> shift)];
    if (page < 0 || page >= c.pages) return nullptr;
    return c.data + (((page * c.kv_heads + head) << shift) + (t & ((1 << shift) - 1))) * Tile<BITS, D>::kBytes;
}

hipError_t launch_cache_append(int bits, int dim, const AppendArgs &a, hipStream_t stream);
hipError_t launch_cache_read(int bits, int dim, const ReadArgs &a, hipStream_t stream);

// The attention's workspace starts with counters, as many whatever the call, so that one workspace
// serves every kernel; parts that are joined follow.
constexpr int kCountersPerCu = 12;
int64_t attention_counter_bytes();

// Few rows a sequence and kv head: one or two operands of 16 columns (256 dimensions: one, for the registers, which is
// what ends it: there is room for no more operands). At that end, 4 kv heads of 64, 128 and 256 dimensions after 500 tokens
// 10.2, 12.8 and 14.8 us and after 32000 tokens 24, 40 and 42; the kernel of many rows takes 18.0, 30.4 and 32.0, and 46, 67
// and 91 for them, and as much for one row more.
constexpr int few_rows(int dim) { return dim == 256 ? 16 : 32; }
int64_t few_workspace(int dim, const AttentionArgs &a);
hipError_t launch_few(int bits, int dim, const AttentionArgs &a, void *workspace, hipStream_t stream);
// Many rows.
int64_t rows_workspace(int dim);
hipError_t launch_rows(int bits, int dim, const AttentionArgs &a, void *workspace, hipStream_t stream);

}  // namespace q8
