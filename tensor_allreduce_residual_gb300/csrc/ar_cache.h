// ar_cache.h -- kernel argument blocks and launcher declarations of the paged
// key-value cache calls, shared by their host side (ar_cache_api.cu) and the
// kernel translation units.
#pragma once

#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ar_internal.h"

namespace ar {

// Strides in elements.
struct AppendArgs {
    const void* q;  // nullable
    const void* k;
    const void* v;
    void* q_out;
    void* k_pages;
    void* v_pages;
    const int* table;
    const int* lengths;
    const int* seq_start;     // nullable: one row per sequence
    const int* positions;     // nullable
    const float* inv_freq;    // nullable with half == 0
    uint64_t q_stride, k_stride, v_stride, q_out_stride;
    uint64_t page_stride, token_stride, head_stride;
    uint64_t capacity;        // max_pages * page_size
    int pages, page_size, table_stride, batch;
    int tokens, q_heads, kv_heads, head_dim;
    int half;                 // rotated pairs of a head
    int interleaved;
    float rotary_scale, k_scale, v_scale;
    int block_tokens;         // rows a block takes: set by the launcher, as are the magics below
    uint64_t turn_magic, row_magic;  // of `half` and of a row's units, used where block_tokens > 1
    int head_units, v_units;  // units of one q or k head, and of one v head
    uint64_t head_magic, v_magic;  // ceil(2^32 / units): u / units == u * magic >> 32 for u * units < 2^32
};

// Rows a block of the append kernel may take, and its threads.
constexpr int kAppendMaxTokens = 8;
constexpr int kAppendThreads = 256;

// One unit is a 16-byte vector of T (vec) or one element, a pair of them where the pair's halves lie apart.
template <typename T, typename CT>
cudaError_t launch_append(const AppendArgs& a, bool vec, cudaStream_t s);

// Strides of the cache in bytes.
struct AttnArgs {
    const char* q;
    const char* k;
    const char* v;
    char* out;
    float* lse;               // nullable
    int2* blocks_of;          // the first and last block of each item
    float* part;              // partial results: two slots per block
    const int* table;
    const int* lengths;
    uint64_t q_stride;        // bytes
    uint64_t page_stride, token_stride, head_stride;
    int table_stride, pages, page_size, batch;
    uint32_t page_magic;      // token / page_size == (2 token * page_magic >> 32) >> page_shift for token < 2^31
    int page_shift;
    int capacity;             // tokens a table row can hold
    int kv_heads, group;      // group: query heads of one key-value head
    int group_blocks;         // the group cut into blocks of at most block_heads
    int block_heads;          // attn_block_heads()
    int head_dim;
    int window;
    float scale2;             // of the scores, k_scale included, in base 2; with softcap twice that over softcap
    float softcap;
    float softcap2;           // softcap in base 2
    float v_scale;
    uint64_t fours_magic;     // x / (head_dim / 4) == x * fours_magic >> 32 for x below 16 * 64
    int slot_floats;          // floats of one partial slot
};

// Query heads of one key-value head that one block attends for at once, at most.  A larger group reads its tiles again for
// every so many: 8 in fp32, whose 16 would not fit a warp's registers with their queries (269 MB at 8 heads 58.6 us, at 16
// 108; bf16 at 16 48.2, at 32 84.4).
__host__ __device__ constexpr int attn_block_heads(int cache_esize) { return cache_esize == 4 ? 8 : 16; }
// Blocks of the attention kernel, at most: three per SM of the 152.  The workspace holds two slots for each.
constexpr int kAttnMaxBlocks = 456;
constexpr int kAttnMaxDim = 256;

// Cached tokens of one tile: what a block loads at once, and the work is cut into.  A warp takes a quarter: 8 tokens in
// fp32; one block of 16 for 16-bit heads over 96; two for those up to 96, and for 8-bit heads of any size.
// 128 tokens against 64, 64 rows of 4096 tokens, 2 key-value heads of 8 query heads each: bf16 heads of 64 26.1
// against 28.0 us; e4m3 heads of 64 21.0 against 24.7, of 128 28.2 against 31.4.  The other way round: bf16 heads of 96 39.5
// against 38.6, with 16 query heads 47.8 against 42.4; e4m3 heads of 192 49.6 against 44.4, of 256 55.0 against 49.6, but of
// 256 with 16 query heads, whose ends of rows fill more than a stage of 64 tokens, 104 against 118.
__host__ __device__ constexpr int attn_tile(int cache_esize, int head_dim)
{
    return cache_esize == 4 ? 32 : cache_esize == 2 && head_dim > 96 ? 64 : 128;
}

// A partial slot: [heads][head_dim] sums, [heads] maxima, [heads] sums of weights.
__host__ __device__ inline int attn_slot_floats(int heads, int head_dim) { return (heads * (head_dim + 2) + 3) / 4 * 4; }

// At most `most` blocks of the attention kernel, and no more than `sms` SMs hold at once; then the join kernel.
template <typename T, typename CT>
cudaError_t launch_attention(const AttnArgs& a, int most, int sms, cudaStream_t s);

struct JoinArgs {
    const void* partials[kMaxRanks];
    const float* lse[kMaxRanks];
    void* out;
    float* lse_out;           // nullable
    int R;
    int dim;                  // elements of a row
    uint64_t elements;        // rows * dim
    uint64_t units;           // threads' worth: set by the launcher
};

// `aligned`: the partials and out are 16-byte aligned.
template <typename T>
cudaError_t launch_join(const JoinArgs& a, bool aligned, cudaStream_t s);

}  // namespace ar
