// ar_tree.h -- kernel arguments of the attention of drafted tokens over a paged
// cache, and what its kernels share with their host side (ar_cache_api.cu).
#pragma once

#include <cuda.h>  // types only: tensor maps are encoded by the driver's function, found at run time
#include <cuda_runtime.h>
#include <stdint.h>

#include "ar_internal.h"

namespace ar {

// Strides of the cache in bytes.
struct TreeArgs {
    const char* q;
    const char* k;
    const char* v;
    char* out;
    float* lse;               // nullable
    struct TreeJob* jobs;     // one for each block: the item it begins and others end
    float* part;              // partial results: two slots per block
    const int* table;
    const int* lengths;
    const int* seq_start;     // nullable: `each` rows a sequence
    const uint32_t* mask;     // nullable: a row sees the drafted tokens up to its own
    uint64_t q_stride;        // bytes
    uint64_t page_stride, token_stride, head_stride;
    int table_stride, pages, page_size, batch;
    uint32_t page_magic;      // token / page_size == (2 token * page_magic >> 32) >> page_shift for token < 2^31
    int page_shift;
    int capacity;             // tokens a table row can hold
    int tokens, each;         // rows of q; of each sequence without seq_start
    int mask_words;           // 32-bit words of a row's mask
    int kv_heads, group, head_dim;
    int window;
    float scale2;             // of the scores, k_scale included, in base 2; with softcap twice that over softcap
    float softcap;
    float softcap2;           // softcap in base 2
    float v_scale;
    int boxes;                // tokens of a tensor copy, 0: pages do not come by them
    int token_first;          // whether the maps' second axis is a page's tokens, and not the heads
    int slot_rows;            // rows of a partial slot: [slot_rows][head_dim] sums, [slot_rows] references, [slot_rows] weights
    uint64_t slot_floats;
    int stall;                // tests only: 1 + the step of k_tree_mma whose weights no warp hands over, so that its waits run out; 0: none
};

// An item that several blocks have parts of, written by the one that begins it; rows == 0: there is none.
struct TreeJob {
    int last;                 // the last block with a part
    int rows;                 // rows of the item
    int first;                // the sequence's first row of q
    int row0;                 // the item's first row in its sequence and head
    int head;                 // key-value head
    int pad[3];
};

// The pages of keys and of values as tensors of elements, tokens and heads (the closer pair first) and pages.
struct TreeMaps {
    CUtensorMap k, v;
};

constexpr int kTreeMaxDim = 256;
// Blocks of the attention kernel, at most: two per SM of the 152.
constexpr int kTreeMaxBlocks = 304;

// Rows of an item (drafted tokens times the query heads of a key-value head) and cached tokens of a tile.
struct TreeShape {
    int rows, tile;
};

// Elements that a head of the matrix kernel has, those of a shorter one followed by zeros.
inline int tree_dim(int head_dim) { return head_dim <= 64 ? 64 : head_dim <= 128 ? 128 : head_dim <= 192 ? 192 : 256; }

// The rule, on what the host knows.  `rows`: of all sequences and one key-value head, padding among them.  An item's cached tokens
// are read once for each block of its rows, so blocks hold the mean item where there is a kernel of that size.  64 sequences of 4096
// tokens, 4 key-value heads of 128 (537 MB of bf16): 32, 64 and 128 rows 137, 141 and 150 us with blocks of 128 and 187, 190 and 204
// with 256; 136 and 256 rows 258 and 265 us with 128 and 203 and 222 with 256.  Heads over 128 leave shared and tensor memory for
// 128 rows only, and tiles of 64 tokens.
// fp32, 16 sequences of 2048 tokens, 8 key-value heads of 96 (201 MB): 10 or 16 rows 140 us with blocks of 16 and 252 with 64, 32
// rows 264 and 253, 64 rows 512 and 258.
inline TreeShape tree_shape(int cache_esize, int head_dim, uint64_t rows, int batch)
{
    if (cache_esize == 4)
        return rows <= 16ull * batch ? TreeShape{16, 32} : TreeShape{64, 32};
    if (head_dim > 128)
        return TreeShape{128, 64};
    return rows <= 128ull * batch ? TreeShape{128, 128} : TreeShape{256, 128};
}

// At most `most` blocks of the attention kernel, and no more than `sms` SMs hold at once; then the join kernel.
template <typename T, typename CT>
cudaError_t launch_tree(const TreeArgs& a, const TreeMaps& maps, const TreeShape& shape, int most, int sms, cudaStream_t s);

// Bounded waits that gave up in the kernels of query type T; the count is cleared.
template <typename T>
cudaError_t take_tree_wait_timeouts(unsigned int* count);

}  // namespace ar
