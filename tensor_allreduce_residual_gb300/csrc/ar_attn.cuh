// ar_attn.cuh -- attention of one new token of each sequence over a paged
// key-value cache.
//
// Work split.  An item is one sequence, one key-value head and its query heads
// (a block of them where they are many); its tokens are cut into tiles.  All items' tiles, in the order
// sequence, head, token, form one line, of which each block takes an equal
// run: blocks finish together whatever the lengths, one long sequence fills
// the GPU as well as many short ones, and the host needs no lengths.  A block
// finds its run by one scan over the lengths.  Rows whose tiles fell to more
// than one block leave a partial sum, maximum and weight in two slots per
// block, which k_attn_join adds up in block order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cfloat>
#include <climits>
#include <type_traits>

#include "ar_cache.h"
#include "ar_kernels.cuh"
#include "ar_launch_k.cuh"
#include "ar_split.h"

namespace ar {

constexpr int kAttnThreads = 128;
constexpr int kAttnWarps = kAttnThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 16-byte asynchronous copies into shared memory; `read` == false writes zeros.  `policy`: how long L2 keeps the line.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void cp_async16_all(uint32_t dst, const void* src, uint64_t policy)
{
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_addr(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Tokens of sequence b: [start, end) are attended to; tile0 is the first tile, tiles how many (at least one, so
// that a row without tokens is written too).
struct Span {
    int start, end, tile0, tiles;
};

template <int TILE>
__device__ __forceinline__ Span span_of_length(const AttnArgs& a, int length)
{
    Span s;
    s.end = min(max(length, 0), a.capacity);
    s.start = a.window > 0 ? max(s.end - a.window, 0) : 0;
    s.tile0 = s.start / TILE;
    s.tiles = max((s.end + TILE - 1) / TILE - s.tile0, 1);
    return s;
}
template <int TILE>
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b)
{
    return span_of_length<TILE>(a, a.lengths[b]);
}

// Where a warp is on the line.  All lanes hold the same, but for `lengths`, of which each has one of 32 sequences'.
struct Cursor {
    int b, hb, tile;  // sequence, head and group block, tile of the item
    Span s;
    uint64_t head_offset;  // of the item's key-value head in a token
    const int* table;      // the sequence's row of the page table
    int lengths, first;    // of sequences first .. first + 31
    __device__ __forceinline__ void load(const AttnArgs& a, int from)
    {
        const int lane = threadIdx.x & 31;
        first = from;
        lengths = from + lane < a.batch ? a.lengths[from + lane] : 0;
    }
    template <int TILE>
    __device__ __forceinline__ void enter(const AttnArgs& a, int sequence)
    {
        b = sequence;
        if (b - first >= 32)
            load(a, b);
        s = span_of_length<TILE>(a, __shfl_sync(~0u, lengths, b - first));
        table = a.table + static_cast<uint64_t>(b) * a.table_stride;
    }
    __device__ __forceinline__ void place(const AttnArgs& a)
    {
        head_offset = static_cast<uint64_t>(a.group_blocks == 1 ? hb : hb / a.group_blocks) * a.head_stride;
    }
    template <int TILE>
    __device__ __forceinline__ void advance(const AttnArgs& a, int heads)
    {
        if (++tile < s.tiles)
            return;
        tile = 0;
        if (++hb == heads) {
            hb = 0;
            enter<TILE>(a, b + 1);
        }
        place(a);
    }
};

// Finds the block's run and its first tile.  All threads; contains barriers.
template <int TILE>
__device__ Run find_run(const AttnArgs& a, int heads, Cursor& cur)
{
    __shared__ long long s_warp[kAttnWarps];
    __shared__ int s_b;
    __shared__ long long s_before;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.batch == 1) {
        cur.load(a, 0);
        cur.enter<TILE>(a, 0);
        const Run run = run_of(static_cast<long long>(cur.s.tiles) * heads, gridDim.x, blockIdx.x);
        cur.hb = static_cast<int>(divide(run.lo, cur.s.tiles));
        cur.tile = static_cast<int>(run.lo - static_cast<long long>(cur.hb) * cur.s.tiles);
        cur.place(a);
        return run;
    }
    // A thread counts the tiles of `per` sequences, all loads at once, and one scan places them on the line: one pass
    // over the lengths, whatever their number (1024 rows of 64 tokens: 15.9 against 17.4 us with scans of 128).
    const int per = (a.batch + kAttnThreads - 1) / kAttnThreads, b0 = tid * per, b1 = min(b0 + per, a.batch);
    long long mine = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b)
        mine += span_of<TILE>(a, b).tiles;
    long long before = mine;  // inclusive, then exclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(~0u, before, o);
        before += lane >= o ? up : 0;
    }
    if (lane == 31)
        s_warp[warp] = before;
    __syncthreads();
    before -= mine;
    long long tiles = 0;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        before += w < warp ? s_warp[w] : 0;
        tiles += s_warp[w];
    }
    const Run run = run_of(tiles * heads, gridDim.x, blockIdx.x);
    if (run.n == 0)
        return run;
    const long long x = divide(run.lo, heads);  // sequence b takes [heads * P, heads * (P + tiles of b)) of the line
    if (before <= x && x < before + mine) {
        int b = b0;
        if (per > 1) {
            for (int n = span_of<TILE>(a, b).tiles; x >= before + n; n = span_of<TILE>(a, b).tiles) {
                before += n;
                ++b;
            }
        }
        s_b = b;
        s_before = before;
    }
    __syncthreads();
    cur.load(a, s_b);
    cur.enter<TILE>(a, s_b);
    const long long in = run.lo - s_before * heads;
    cur.hb = static_cast<int>(divide(in, cur.s.tiles));
    cur.tile = static_cast<int>(in - static_cast<long long>(cur.hb) * cur.s.tiles);
    cur.place(a);
    return run;
}

// Row of the output of head `i` of the item's group block, and how many heads the block has.
__device__ __forceinline__ uint64_t out_row(const AttnArgs& a, int b, int hb, int i)
{
    const int h = a.group_blocks == 1 ? hb : hb / a.group_blocks, gb = hb - h * a.group_blocks;
    return (static_cast<uint64_t>(b) * a.kv_heads + h) * a.group + gb * a.block_heads + i;
}
__device__ __forceinline__ int heads_of(const AttnArgs& a, int hb)
{
    return a.group_blocks == 1 ? a.group : min(a.group - (hb % a.group_blocks) * a.block_heads, a.block_heads);
}

__device__ __forceinline__ float lse_of(float top2, float total)
{
    return total == 0.0f ? -INFINITY : (top2 + log2f(total)) * kLn2;
}
// What sums of weighted values are multiplied by.
__device__ __forceinline__ float out_scale(const AttnArgs& a, float total)
{
    return total == 0.0f ? 0.0f : a.v_scale / total;
}

// 2^x, off by 2^-22 of it at the most, less than a pair of 16-bit numbers leaves of a weight.  Results under 2^-126, which
// no sum of weights from 1 on shows, are 0.
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// tanh(x) of 2 x in base 2, off by 2^-20 of it at the most, so that a softcap far above the scores leaves them as they are:
// (e - 1) / (e + 1) with e = e^(2 x), and below 0.3, where e - 1 would lose bits, five terms of the series.
__device__ __forceinline__ float tanh_fast(float two_x)
{
    const float e = exp2_fast(two_x > 64.0f ? 64.0f : two_x);  // a NaN stays one
    const float x = two_x * (0.5f * kLn2), y = x * x;
    const float series = fmaf(fmaf(fmaf(fmaf(62.0f / 2835.0f, y, -17.0f / 315.0f), y, 2.0f / 15.0f), y, -1.0f / 3.0f), y * x, x);
    return fabsf(x) < 0.3f ? series : __fdividef(e - 1.0f, e + 1.0f);
}
// What a maximum is subtracted as: minus infinity stands for no token yet, and 0 in its place keeps differences defined.
__device__ __forceinline__ float base_of(float top) { return top == -INFINITY ? 0.0f : top; }

// Four elements of a row of the output.
template <typename T>
__device__ __forceinline__ void store_four(T* out, float4 v, float f)
{
    if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(out) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
    else
        *reinterpret_cast<uint2*>(out) = make_uint2(Lanes<T>::word(v.x * f, v.y * f), Lanes<T>::word(v.z * f, v.w * f));
}

// ---------------------------------------------------------------------------
// Shape of an attention kernel: query type, cache type, head elements (those
// of a shorter head are followed by zeros) and query heads of a block.
//
// Each warp takes a quarter of a tile's tokens, through a ring of stages of its
// own filled by asynchronous 16-byte copies, with a maximum, a sum and an
// accumulator of its own.  The four warps meet at the ends of the block's part
// of an item only; between them no warp waits for another.
// ---------------------------------------------------------------------------
template <typename T_, typename CT_, int DIM_, int HEADS_>
struct AttnShape {
    using T = T_;
    using CT = CT_;
    static constexpr int DIM = DIM_, HEADS = HEADS_;
    static constexpr bool SMALL = sizeof(CT) == 1, WIDE = sizeof(CT) == 4;
    static constexpr int TILE = attn_tile(sizeof(CT), DIM);
    static constexpr int TOKENS = TILE / kAttnWarps;  // a warp's tokens of a tile
    static constexpr int CHUNKS = DIM * sizeof(CT) / 16;
    static constexpr int QCHUNKS = DIM * sizeof(T) / 16;
    // 16-byte chunks of a row: permuted within 128 bytes by the row, or padded to an odd number; either way the eight
    // rows of an 8 x 8 matrix lie in different banks.
    static constexpr int PITCH = CHUNKS % 8 == 0 ? CHUNKS : CHUNKS | 1;
    static constexpr int QPITCH = QCHUNKS % 8 == 0 ? QCHUNKS : QCHUNKS | 1;
    static constexpr int HALF = TOKENS * PITCH * 16;     // a warp's keys of a stage, and its values
    static constexpr int QROWS = kAttnWarps * 2 * HALF;  // where a stage's queries begin
    static constexpr int STAGE = QROWS + HEADS * QPITCH * 16;
    static constexpr int INFO = kAttnWarps * (TOKENS * 8 + 16);
    // Shared memory of a block besides: the fp32 kernel's weights of a tile.
    static constexpr int OTHER = WIDE ? (TILE + kAttnWarps) * HEADS * 4 : 0;
    static constexpr int OPITCH = DIM + 4;  // floats; the epilogue's rows, one per warp and head, lie in a used stage
    static_assert(kAttnWarps * HEADS * OPITCH * 4 <= STAGE, "the epilogue fits a stage");
    static_assert(STAGE % 128 == 0 && (CHUNKS % 8 != 0 || HALF % 128 == 0), "permuted rows begin at multiples of 128 bytes");
    static constexpr int fits(int bytes)
    {
        const int n = (bytes - kSmemReservedPerBlock - 1024 - INFO - OTHER) / (STAGE + INFO);
        return n < 5 ? n : 5;
    }
    // Blocks of an SM: three where registers and two stages of each fit, which short rows and 8-bit elements gain from most
    // (256 rows of 1 to 200 tokens, 8 key-value heads of 128 bf16 elements: 37.8 against 45.9 us with two; 511 MB of them in
    // longer rows: 83.9 against 84.7; 533 MB of e4m3: 86.1 against 90.4; 93 MB of fp16 heads of 64: 21.7 against 24.3); two
    // for stages over 48 KB or where a block of 8 or 16 heads needs the registers of a third.  One where the shared memory
    // has no room for two stages of each: heads over 192, over 128 in 8 bits, of 72 to 96 in 16 bits with more than 8 query
    // heads, and over 128 in fp32 with one or two (of those, 129 to 192 would fit two blocks).
    static constexpr int WANT = HEADS == 2 || (HEADS == 8 && DIM <= 128 && STAGE < 48 * 1024 && (!WIDE || DIM <= 64)) ? 3 : 2;
    static constexpr int BLOCKS = fits(kSmemPerSM / WANT) >= 2 ? WANT : 1;
    static constexpr int STAGES = fits(kSmemPerSM / BLOCKS);
    static constexpr int RING = STAGES + 1;  // descriptions of tiles: one more is written than copies are under way
    static constexpr int SMEM = STAGES * STAGE;
    static __device__ __forceinline__ int chunk(int row, int c)
    {
        return CHUNKS % 8 == 0 ? row * PITCH + (c ^ (row & 7)) : row * PITCH + c;
    }
    static __device__ __forceinline__ int qchunk(int row, int c)
    {
        return QCHUNKS % 8 == 0 ? row * QPITCH + (c ^ (row & 7)) : row * QPITCH + c;
    }
};

// A warp's part of one tile in flight: whose it is, its tokens' offsets in the cache, and which of them count.
enum { kTileFirst = 1, kTileLast = 2, kTileBegins = 4, kTileEnds = 8 };  // of the block's part; of the item
template <int TOKENS>
struct WarpTile {
    long long offset[TOKENS];
    int b, hb, flags;
    uint32_t in;
};

// A warp's ring: describes the tiles of the block's run one after the other, and issues the copies of described ones.
template <typename P>
struct Feed {
    using Tile = WarpTile<P::TOKENS>;
    const AttnArgs& a;
    Tile* tiles;  // [RING]
    char* smem;
    int heads, n, warp, lane, chunks, qchunks;
    Cursor cur;
    uint64_t policy;
    int described = 0, ring_w = 0, ring_i = P::STAGES - 1, ring_r = 0, stage_w = P::STAGES - 1, stage_r = 0;

    __device__ Feed(const AttnArgs& a_, Tile* tiles_, char* smem_, int n_, const Cursor& c)
        : a(a_), tiles(tiles_), smem(smem_), heads(a_.kv_heads * a_.group_blocks), n(n_), warp(threadIdx.x >> 5), lane(threadIdx.x & 31),
          chunks(a_.head_dim * static_cast<int>(sizeof(typename P::CT)) / 16), qchunks(a_.head_dim * static_cast<int>(sizeof(typename P::T)) / 16),
          cur(c)
    {
        // The cache streams through L2 and leaves it to others, unless more query heads are to read the same tiles.
        // (511 MB of bf16 cache: 87.1 against 89.8 us; 67 MB: 18.0 against 19.0.)
        if (a.group_blocks == 1)
            asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
        else
            asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(policy));
    }

    // The next tile's description, in two steps, with its pages' numbers on their way between them.
    struct Pending {
        int page = -1, slot = 0;
        uint64_t head_offset;
        Tile* tile = nullptr;
    } pending;
    __device__ __forceinline__ void open(Pending& p)
    {
        p.tile = nullptr;
        if (described >= n)
            return;
        p.tile = &tiles[ring_w];
        const int token = (cur.s.tile0 + cur.tile) * P::TILE + warp * P::TOKENS + lane;
        p.page = -1;
        if (lane < P::TOKENS && token >= cur.s.start && token < cur.s.end) {
            const uint32_t column = __umulhi(2u * token, a.page_magic) >> a.page_shift;
            p.slot = token - static_cast<int>(column) * a.page_size;
            p.page = cur.table[column];
        }
        p.head_offset = cur.head_offset;
        if (lane == 0) {
            const bool begins = cur.tile == 0, ends = cur.tile + 1 == cur.s.tiles;
            p.tile->b = cur.b;
            p.tile->hb = cur.hb;
            p.tile->flags = (begins || described == 0 ? kTileFirst : 0) | (ends || described + 1 == n ? kTileLast : 0) |
                            (begins ? kTileBegins : 0) | (ends ? kTileEnds : 0);
        }
        ++described;
        ring_w = ring_w + 1 == P::RING ? 0 : ring_w + 1;
        if (described < n)
            cur.advance<P::TILE>(a, heads);
    }
    __device__ __forceinline__ void close(const Pending& p)
    {
        if (p.tile == nullptr)
            return;
        const bool in = p.page >= 0 && p.page < a.pages;
        const uint32_t mask = __ballot_sync(~0u, in);
        if (lane < P::TOKENS)
            p.tile->offset[lane] = in ? static_cast<long long>(static_cast<uint32_t>(p.page) * a.page_stride +
                                                               static_cast<uint32_t>(p.slot) * a.token_stride + p.head_offset)
                                      : 0;
        if (lane == 0)
            p.tile->in = mask;
    }
    // The warp's copies of a described tile, and its share of a new item's queries.  Chunks beyond the head's elements
    // and tokens that are left out become zeros.
    __device__ __forceinline__ void issue(const Tile& tile, int stage)
    {
        const uint32_t base = smem_addr(smem + stage * P::STAGE);
        const uint32_t ks = base + warp * 2 * P::HALF;
        const uint32_t in = tile.in;
        constexpr uint32_t ALL = P::TOKENS == 32 ? ~0u : (1u << P::TOKENS) - 1;
        if (in == ALL && chunks == P::CHUNKS) {
            // 32 lanes cover PER * 32 chunks, ROWS whole rows, in PER steps; then everything repeats ROWS rows further, where
            // the rows' permutation flips address bits 4 to 6 by a constant.
            constexpr int ROWS = P::CHUNKS % 32 == 0 ? 1 : P::CHUNKS % 16 == 0 ? 2 : P::CHUNKS % 8 == 0 ? 4 : P::CHUNKS % 4 == 0 ? 8 : 16;
            constexpr int PER = ROWS * P::CHUNKS / 32;
            static_assert(PER * 32 == ROWS * P::CHUNKS && P::TOKENS % ROWS == 0, "whole rows, whole tiles");
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int row0 = (lane + 32 * j) / P::CHUNKS, c = lane + 32 * j - row0 * P::CHUNKS;
                const char* const k = a.k + c * 16;
                const char* const v = a.v + c * 16;
                const uint32_t first = ks + P::chunk(row0, c) * 16;
#pragma unroll
                for (int i = 0; i < P::TOKENS; i += ROWS) {
                    const long long at = tile.offset[row0 + i];
                    const uint32_t flip = P::CHUNKS % 8 == 0 ? (i & 7) << 4 : 0;
                    const uint32_t dst = (first ^ flip) + i * P::PITCH * 16;
                    cp_async16_all(dst, k + at, policy);
                    cp_async16_all(dst + P::HALF, v + at, policy);
                }
            }
        } else {
#pragma unroll 4
            for (int i = 0; i < P::TOKENS * P::CHUNKS / 32; ++i) {
                const int row = (lane + i * 32) / P::CHUNKS, c = lane + i * 32 - row * P::CHUNKS;
                const bool read = (in >> row & 1) != 0 && c < chunks;
                const long long at = tile.offset[row] + (c < chunks ? c * 16 : 0);
                const uint32_t dst = ks + P::chunk(row, c) * 16;
                cp_async16(dst, a.k + at, read, policy);
                cp_async16(dst + P::HALF, a.v + at, read, policy);
            }
        }
        if (tile.flags & kTileFirst) {
            const int g = heads_of(a, tile.hb);
            const char* q = a.q + tile.b * a.q_stride + out_row(a, 0, tile.hb, 0) * a.head_dim * sizeof(typename P::T);
            for (int x = threadIdx.x; x < P::HEADS * P::QCHUNKS; x += kAttnThreads) {
                const int row = x / P::QCHUNKS, c = x - row * P::QCHUNKS;
                const bool read = row < g && c < qchunks;
                cp_async16(base + P::QROWS + P::qchunk(row, c) * 16,
                           q + (read ? static_cast<size_t>(row) * a.head_dim * sizeof(typename P::T) + c * 16 : 0), read);
            }
        }
    }
    // Fills the ring before the first tile.
    __device__ __forceinline__ void start()
    {
        Pending p[P::STAGES];
#pragma unroll
        for (int i = 0; i < P::STAGES; ++i)
            open(p[i]);
#pragma unroll
        for (int i = 0; i < P::STAGES; ++i) {
            close(p[i]);
            __syncwarp();
            if (i + 1 < P::STAGES) {
                if (i < n)
                    issue(tiles[i], i);
                cp_async_commit();
            }
        }
    }
    // Waits for tile t's copies and sends the next ones on their way.
    __device__ __forceinline__ void turn(int t)
    {
        cp_async_wait<P::STAGES - 2>();
        __syncwarp();
        if (t + P::STAGES - 1 < n)
            issue(tiles[ring_i], stage_w);
        cp_async_commit();
        open(pending);
    }
    __device__ __forceinline__ void next()
    {
        close(pending);
        ring_r = ring_r + 1 == P::RING ? 0 : ring_r + 1;
        ring_i = ring_i + 1 == P::RING ? 0 : ring_i + 1;
        stage_r = stage_r + 1 == P::STAGES ? 0 : stage_r + 1;
        stage_w = stage_w + 1 == P::STAGES ? 0 : stage_w + 1;
    }
};

// The end of the block's part of an item, after every warp has left its maxima, sums (s_top, s_total) and accumulators,
// the latter scaled to the block's maximum, in `rows`: adds the warps' up and writes the result or the part.  `first`: the
// run's tile that this part began with.
template <typename P>
__device__ __forceinline__ void write_part(const AttnArgs& a, const WarpTile<P::TOKENS>& tile, const Run& run, int first, bool began,
                                           const float* rows, const float (*s_top)[P::HEADS], const float (*s_total)[P::HEADS])
{
    using T = typename P::T;
    const bool whole = began && (tile.flags & kTileEnds);
    const int g = heads_of(a, tile.hb), fours = a.head_dim / 4, slots = min(a.group, a.block_heads);
    float* part = a.part + slot_of(static_cast<int>(blockIdx.x), began) * a.slot_floats;
    if (began && threadIdx.x == 0) {  // tells the join which blocks have the item's parts
        int last = static_cast<int>(blockIdx.x);
        if (!whole)
            last = block_of(run.total, static_cast<int>(gridDim.x), run.lo + first + span_of<P::TILE>(a, tile.b).tiles - 1);
        a.blocks_of[static_cast<uint64_t>(tile.b) * (a.kv_heads * a.group_blocks) + tile.hb] = make_int2(static_cast<int>(blockIdx.x), last);
    }
    for (int x = threadIdx.x; x < g * fours; x += kAttnThreads) {
        const int head = static_cast<int>(static_cast<uint32_t>(x) * a.fours_magic >> 32), d = (x - head * fours) * 4;
        float best = s_top[0][head], sum = 0.0f;
#pragma unroll
        for (int w = 1; w < kAttnWarps; ++w)
            best = fmaxf(best, s_top[w][head]);
        const float base = base_of(best);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            sum += s_total[w][head] * exp2_fast(s_top[w][head] - base);
            const float4 y = *reinterpret_cast<const float4*>(rows + (w * P::HEADS + head) * P::OPITCH + d);
            v.x += y.x;
            v.y += y.y;
            v.z += y.z;
            v.w += y.w;
        }
        if (whole) {
            const uint64_t row = out_row(a, tile.b, tile.hb, head);
            store_four(reinterpret_cast<T*>(a.out) + row * a.head_dim + d, v, out_scale(a, sum));
            if (d == 0 && a.lse != nullptr)
                a.lse[row] = lse_of(best, sum);
        } else {
            *reinterpret_cast<float4*>(part + head * a.head_dim + d) = v;
            if (d == 0) {
                part[slots * a.head_dim + head] = best;
                part[slots * (a.head_dim + 1) + head] = sum;
            }
        }
    }
}

// a * b + c of two numbers at once.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

// Maximum or sum over the eight lanes that differ in the lane's upper three bits.
__device__ __forceinline__ float column_max(float x)
{
#pragma unroll
    for (int w = 4; w < 32; w <<= 1)
        x = fmaxf(x, __shfl_xor_sync(~0u, x, w));
    return x;
}
__device__ __forceinline__ float column_sum(float x)
{
#pragma unroll
    for (int w = 4; w < 32; w <<= 1)
        x += __shfl_xor_sync(~0u, x, w);
    return x;
}

// ---------------------------------------------------------------------------
// The fp32 kernel: multiply-adds, as no matrix instruction keeps 24 bits.  A
// lane has four elements of the head (eight of the longest), of the queries in
// registers, and forms its part of every token's and head's product; then the
// lanes halve what they hold in five exchanges, each keeping and receiving a
// half, and end with one token's sums for a quarter of the heads.  So a cached
// element is read from shared memory once, and no query is.  (Four lanes a
// token, the queries in shared memory, read those four times as often as the
// cache: 68 us on 269 MB with 8 heads, its loads at 64 % of the pipe.)  For the
// weighted values the same elements take every token's weights, from shared
// memory.  Heads of up to 64 elements take half of the lanes, and each half
// half of the tokens.  With 8 query heads of more than 128 elements it spills
// 80 to 148 bytes a thread (0.67 of the copy rate, as at 128 without).
// ---------------------------------------------------------------------------
template <typename P>
__global__ void __launch_bounds__(kAttnThreads, P::BLOCKS)
k_attn_fma(const AttnArgs a)
{
    constexpr int HEADS = P::HEADS, COLS = P::DIM / 4, CPL = (COLS + 31) / 32, HALVES = COLS <= 16 ? 2 : 1;
    constexpr int HL = HEADS >= 4 ? HEADS / 4 : 1;  // heads whose sums a lane ends with
    constexpr int MINE = P::TOKENS / HALVES;        // tokens a lane has a part of
    static_assert(P::TOKENS == 8, "eight tokens by four quarters of the heads");
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(16) WarpTile<P::TOKENS> s_tiles[kAttnWarps][P::RING];
    __shared__ float s_top[kAttnWarps][HEADS], s_total[kAttnWarps][HEADS];
    __shared__ __align__(16) float s_weights[kAttnWarps][(P::TOKENS + 1) * HEADS];  // [TOKENS][HEADS], then [HEADS] factors
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float* const s_p = s_weights[warp];
    float* const s_fix = s_p + P::TOKENS * HEADS;

    Cursor cur;
    const Run run = find_run<P::TILE>(a, a.kv_heads * a.group_blocks, cur);
    if (run.n == 0)
        return;
    Feed<P> feed(a, s_tiles[warp], smem, static_cast<int>(min(run.n, static_cast<long long>(INT_MAX))), cur);
    feed.start();

    const int quarter = lane & 3, token = lane >> 2;
    const int head0 = HEADS >= 4 ? quarter * HL : quarter >> 1;
    const int col = HALVES == 2 ? lane & 15 : lane, row0 = HALVES == 2 ? (lane >> 4) * MINE : 0;
    const auto has = [&](int c) { return COLS % 32 == 0 || HALVES == 2 || col + 32 * c < COLS; };
    float4 q[HEADS][CPL], o[HEADS][CPL];
    float top[HL], total[HL];
    bool began = false;  // whether the block's part of the item begins it
    int first = 0;       // the part's first tile
#pragma unroll 1
    for (int t = 0; t < feed.n; ++t) {
        feed.turn(t);
        const WarpTile<P::TOKENS>& tile = feed.tiles[feed.ring_r];
        const int flags = tile.flags;
        char* const stage = smem + feed.stage_r * P::STAGE;
        const char* const ks = stage + warp * 2 * P::HALF;
        const char* const vs = ks + P::HALF;
        if (flags & kTileFirst) {
            began = flags & kTileBegins;
            first = t;
            __syncthreads();  // the queries are the block's
#pragma unroll
            for (int h = 0; h < HEADS; ++h)
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    q[h][c] = o[h][c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (has(c))
                        q[h][c] = *reinterpret_cast<const float4*>(stage + P::QROWS + P::qchunk(h, col + 32 * c) * 16);
                }
#pragma unroll
            for (int i = 0; i < HL; ++i) {
                top[i] = -INFINITY;
                total[i] = 0.0f;
            }
            __syncthreads();  // a warp ahead may bring the next queries here
        }

        float dot[MINE * HEADS];
#pragma unroll
        for (int j = 0; j < MINE; ++j) {
            float4 k[CPL];
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                k[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (has(c))
                    k[c] = *reinterpret_cast<const float4*>(ks + P::chunk(row0 + j, col + 32 * c) * 16);
            }
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                float2 x = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    x = fma2(make_float2(q[h][c].x, q[h][c].y), make_float2(k[c].x, k[c].y), x);
                    x = fma2(make_float2(q[h][c].z, q[h][c].w), make_float2(k[c].z, k[c].w), x);
                }
                dot[j * HEADS + h] = x.x + x.y;
            }
        }
        // Lane bits 4 to 2 choose the token (bit 4 does already where it chooses the half), bits 1 and 0 the heads.
        int held = MINE * HEADS;
#pragma unroll
        for (int w = 16 / HALVES; w > 0; w >>= 1) {
            if (held > 1) {
                held /= 2;
#pragma unroll
                for (int i = 0; i < MINE * HEADS / 2; ++i)
                    if (i < held) {
                        const float keep = lane & w ? dot[i + held] : dot[i], send = lane & w ? dot[i] : dot[i + held];
                        dot[i] = keep + __shfl_xor_sync(~0u, send, w);
                    }
            } else {
                dot[0] += __shfl_xor_sync(~0u, dot[0], w);
            }
        }
        const bool in = (tile.in >> token & 1) != 0;
        bool moved = false;
        float fix[HL];
#pragma unroll
        for (int i = 0; i < HL; ++i) {
            float x = dot[i] * a.scale2;
            if (a.softcap > 0.0f)
                x = a.softcap2 * tanhf(x * (0.5f * kLn2));
            x = in ? x : -INFINITY;
            const float best = fmaxf(column_max(x), top[i]);
            moved = moved || best > top[i];
            fix[i] = exp2f(top[i] - base_of(best));
            const float p = exp2f(x - base_of(best));
            total[i] = total[i] * fix[i] + p;
            top[i] = best;
            if (HEADS >= 4 || (quarter & 1) == 0)
                s_p[token * HEADS + head0 + i] = p;
        }
        if (__any_sync(~0u, moved)) {
            if (token == 0 && (HEADS >= 4 || (quarter & 1) == 0)) {
#pragma unroll
                for (int i = 0; i < HL; ++i)
                    s_fix[head0 + i] = fix[i];
            }
            __syncwarp();
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                const float f = s_fix[h];
#pragma unroll
                for (int c = 0; c < CPL; ++c)
                    o[h][c] = make_float4(o[h][c].x * f, o[h][c].y * f, o[h][c].z * f, o[h][c].w * f);
            }
        }
        __syncwarp();
#pragma unroll
        for (int j = 0; j < MINE; ++j) {
            const int row = row0 + j;
            float p[HEADS];
            if constexpr (HEADS >= 4) {
#pragma unroll
                for (int h = 0; h < HEADS; h += 4)
                    *reinterpret_cast<float4*>(p + h) = *reinterpret_cast<const float4*>(s_p + row * HEADS + h);
            } else {
                *reinterpret_cast<float2*>(p) = *reinterpret_cast<const float2*>(s_p + row * HEADS);
            }
#pragma unroll
            for (int c = 0; c < CPL; ++c) {
                if (has(c)) {
                    const float4 v = *reinterpret_cast<const float4*>(vs + P::chunk(row, col + 32 * c) * 16);
#pragma unroll
                    for (int h = 0; h < HEADS; ++h) {
                        const float2 two = make_float2(p[h], p[h]);
                        const float2 x = fma2(two, make_float2(v.x, v.y), make_float2(o[h][c].x, o[h][c].y));
                        const float2 y = fma2(two, make_float2(v.z, v.w), make_float2(o[h][c].z, o[h][c].w));
                        o[h][c] = make_float4(x.x, x.y, y.x, y.y);
                    }
                }
            }
        }

        if (flags & kTileLast) {
#pragma unroll
            for (int i = 0; i < HL; ++i) {
                const float sum = column_sum(total[i]);
                if (token == 0 && (HEADS >= 4 || (quarter & 1) == 0)) {
                    s_top[warp][head0 + i] = top[i];
                    s_total[warp][head0 + i] = sum;
                }
            }
            __syncthreads();  // and every warp is done with the stage
            float* const rows = reinterpret_cast<float*>(stage);
#pragma unroll
            for (int h = 0; h < HEADS; ++h) {
                float best = s_top[0][h];
#pragma unroll
                for (int w = 1; w < kAttnWarps; ++w)
                    best = fmaxf(best, s_top[w][h]);
                const float f = exp2_fast(s_top[warp][h] - base_of(best));
#pragma unroll
                for (int c = 0; c < CPL; ++c) {
                    float4 v = o[h][c];
                    if constexpr (HALVES == 2) {
                        v.x += __shfl_xor_sync(~0u, v.x, 16);
                        v.y += __shfl_xor_sync(~0u, v.y, 16);
                        v.z += __shfl_xor_sync(~0u, v.z, 16);
                        v.w += __shfl_xor_sync(~0u, v.w, 16);
                    }
                    if (COLS % 32 == 0 || (HALVES == 2 ? lane < 16 : col + 32 * c < COLS))
                        *reinterpret_cast<float4*>(rows + (warp * HEADS + h) * P::OPITCH + (col + 32 * c) * 4) =
                            make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
                }
            }
            __syncthreads();
            write_part<P>(a, tile, run, first, began, rows, s_top, s_total);
            __syncthreads();  // the next copies go to this stage
        }
        feed.next();
    }
}

// ---------------------------------------------------------------------------
// The matrix kernel, for 16-bit and 8-bit caches.  Scores are computed as
// K Q^T and values as V^T P^T: tokens, and then the head's elements, are the
// 16 rows of a matrix instruction and query heads its 8 columns, so that up to
// 8 heads fill it where rows of queries would leave half of it empty, and both
// operands from the cache come out of shared memory by ldmatrix as they lie
// there.  Weights enter the second product as a pair of 16-bit numbers, their
// rounding and what it leaves (17 bits and more together), which costs an
// instruction that the memory's pace hides (bf16 queries on 533 MB of e4m3:
// 85.6 us, with the first number alone 85.1; 16 heads of 128 on 134 MB: 37.0
// against 34.0).  8-bit elements become fp16 in registers, exactly; queries too
// large or small for fp16 are scaled by a power of two per head first.  The
// kernels of 16 query heads of 256 elements spill 68 bytes a thread in 16 bits
// and about 400 in 8 (0.53 and 0.36 of the copy rate).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t* r)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t* r)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
template <typename MT>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<MT, __half>::value)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 values of the lower 16 bits as fp16, exactly.
__device__ __forceinline__ uint32_t half2_of_e4m3(uint32_t x)
{
    uint32_t y;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(y) : "h"(static_cast<uint16_t>(x)));
    return y;
}
template <typename P>
__global__ void __launch_bounds__(kAttnThreads, P::BLOCKS)
k_attn_mma(const AttnArgs a)
{
    using T = typename P::T;
    using MT = typename std::conditional<P::SMALL, __half, typename P::CT>::type;  // of the instructions' operands
    constexpr int TOKENS = P::TOKENS, KB = TOKENS / 16, NT = P::HEADS / 8, MTILES = P::DIM / 16, KSTEPS = P::DIM / 16;
    // Weights in fp16 are 2^15 times as large, the largest 2^15: those down to 2^-29 of it keep all their bits, and thousands
    // of small ones do not vanish beside a few large.
    constexpr float LIFT = std::is_same<MT, __half>::value ? 0x1p15f : 1.0f;
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(16) WarpTile<TOKENS> s_tiles[kAttnWarps][P::RING];
    __shared__ float s_top[kAttnWarps][P::HEADS], s_total[kAttnWarps][P::HEADS];
    pdl_enter();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g8 = lane >> 2, t4 = lane & 3;

    Cursor cur;
    const Run run = find_run<P::TILE>(a, a.kv_heads * a.group_blocks, cur);
    if (run.n == 0)
        return;
    Feed<P> feed(a, s_tiles[warp], smem, static_cast<int>(min(run.n, static_cast<long long>(INT_MAX))), cur);
    feed.start();

    uint32_t qf[NT][KSTEPS][2];
    float o[NT][MTILES][4], top[NT][2], total[NT][2], qscale[NT][2];
    bool began = false;  // whether the block's part of the item begins it
    int first = 0;       // the part's first tile
#pragma unroll 1
    for (int t = 0; t < feed.n; ++t) {
        feed.turn(t);
        const WarpTile<TOKENS>& tile = feed.tiles[feed.ring_r];
        const int flags = tile.flags;
        char* stage = smem + feed.stage_r * P::STAGE;
        const uint32_t ks = smem_addr(stage) + warp * 2 * P::HALF, vs = ks + P::HALF, qs = smem_addr(stage) + P::QROWS;
        if (flags & kTileFirst)
            __syncthreads();  // the queries are the block's
        if (flags & kTileFirst) {
            began = flags & kTileBegins;
            first = t;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if constexpr (!P::SMALL) {
#pragma unroll
                    for (int j = 0; j < KSTEPS; j += 2)
                        ldmatrix4(qs + P::qchunk(nt * 8 + (lane & 7), 2 * j + (lane >> 3)) * 16, &qf[nt][j][0]);
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        qscale[nt][i] = a.scale2;
                } else {
                    // Elements 4 t4 .. 4 t4 + 3 of each 16: the order in which the 8-bit keys' come.
                    float most = 0.0f;
#pragma unroll
                    for (int j = 0; j < KSTEPS; ++j) {
                        const uint2 w = *reinterpret_cast<const uint2*>(
                            stage + P::QROWS + P::qchunk(nt * 8 + g8, 2 * j + (t4 >> 1)) * 16 + (t4 & 1) * 8);
                        qf[nt][j][0] = w.x;
                        qf[nt][j][1] = w.y;
                        if constexpr (!std::is_same<T, __half>::value) {
                            const float2 x = Lanes<T>::two(w.x), y = Lanes<T>::two(w.y);
                            most = fmaxf(most, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
                        }
                    }
                    // The largest element becomes 2^14 or more: elements down to 2^-28 of it keep all their bits.  (Scaled to 1, those
                    // under 2^-25 of it would vanish.)
                    int e = 0;
                    if constexpr (!std::is_same<T, __half>::value) {
                        most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
                        most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
                        e = max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -112) - 14;
                        const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                        for (int j = 0; j < KSTEPS; ++j)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float2 x = Lanes<T>::two(qf[nt][j][i]);
                                qf[nt][j][i] = Lanes<__half>::word(x.x * down, x.y * down);
                            }
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int eh = __shfl_sync(~0u, e, (2 * t4 + i) * 4);
                        // Finite: an infinite factor would make the scores of keys that are 0 NaN.
                        qscale[nt][i] = fmaxf(fminf(ldexpf(a.scale2, eh), FLT_MAX), -FLT_MAX);
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    top[nt][i] = -INFINITY;
                    total[nt][i] = 0.0f;
                }
#pragma unroll
                for (int m = 0; m < MTILES; ++m)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        o[nt][m][i] = 0.0f;
            }
            __syncthreads();  // a warp ahead may bring the next queries here
        }

        // Scores of the warp's tokens: rows g8 and g8 + 8 of each block, heads 2 t4 and 2 t4 + 1 of each eight.  Two sums
        // each, of even and odd steps, so that an instruction need not wait for the one before.
        float s[KB][NT][4];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int row = kb * 16 + (lane & 15);
            float odd[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[kb][nt][i] = odd[nt][i] = 0.0f;
#pragma unroll
            for (int j = 0; j < P::CHUNKS / 2; ++j) {
                uint32_t r[4];
                ldmatrix4(ks + P::chunk(row, 2 * j + (lane >> 4)) * 16, r);
                if constexpr (!P::SMALL) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816<MT>(j % 2 == 0 ? s[kb][nt] : odd[nt], r, qf[nt][j][0], qf[nt][j][1]);
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t k[4] = {half2_of_e4m3(r[2 * c]), half2_of_e4m3(r[2 * c + 1]),
                                               half2_of_e4m3(r[2 * c] >> 16), half2_of_e4m3(r[2 * c + 1] >> 16)};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<MT>(c == 0 ? s[kb][nt] : odd[nt], k, qf[nt][2 * j + c][0], qf[nt][2 * j + c][1]);
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s[kb][nt][i] = (s[kb][nt][i] + odd[nt][i]) * qscale[nt][i & 1];
        }
        if (a.softcap > 0.0f) {
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[kb][nt][i] = a.softcap2 * tanh_fast(s[kb][nt][i]);
        }
        if (tile.in != (TOKENS == 32 ? ~0u : 0xffffu)) {
            const uint32_t in = tile.in >> g8;
#pragma unroll
            for (int kb = 0; kb < KB; ++kb)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        s[kb][nt][i] = (in >> (kb * 16 + (i < 2 ? 0 : 8)) & 1) != 0 ? s[kb][nt][i] : -INFINITY;
        }

        // The running maximum and sum.
        uint32_t hi[KB][NT][2], lo[KB][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float base[2];
            bool moved = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = fmaxf(s[0][nt][i], s[0][nt][i + 2]);
#pragma unroll
                for (int kb = 1; kb < KB; ++kb)
                    x = fmaxf(x, fmaxf(s[kb][nt][i], s[kb][nt][i + 2]));
                x = fmaxf(column_max(x), top[nt][i]);
                moved = moved || x > top[nt][i];
                base[i] = x;
            }
            if (__any_sync(~0u, moved)) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float fix = exp2_fast(top[nt][i] - base_of(base[i]));
                    top[nt][i] = base[i];
                    total[nt][i] *= fix;
#pragma unroll
                    for (int m = 0; m < MTILES; ++m) {
                        o[nt][m][i] *= fix;
                        o[nt][m][i + 2] *= fix;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                base[i] = base_of(base[i]);
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float p0 = exp2_fast(s[kb][nt][2 * r] - base[0]);
                    const float p1 = exp2_fast(s[kb][nt][2 * r + 1] - base[1]);
                    total[nt][0] += p0;
                    total[nt][1] += p1;
                    const uint32_t h = Lanes<MT>::word(p0 * LIFT, p1 * LIFT);
                    hi[kb][nt][r] = transposed(h);
                    const float2 back = Lanes<MT>::two(h);
                    lo[kb][nt][r] = transposed(Lanes<MT>::word(fmaf(p0, LIFT, -back.x), fmaf(p1, LIFT, -back.y)));
                }
            }
        }

        // Weighted values.  Rows of the result: elements g8 and g8 + 8 of each 16, or 2 g8 and 2 g8 + 1 (8-bit).
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
            const int row = kb * 16;
            if constexpr (!P::SMALL) {
#pragma unroll
                for (int m = 0; m < MTILES; ++m) {
                    uint32_t r[4];
                    ldmatrix4_trans(vs + P::chunk(row + (lane & 7) + (lane >> 4) * 8, 2 * m + (lane >> 3 & 1)) * 16, r);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816<MT>(o[nt][m], r, hi[kb][nt][0], hi[kb][nt][1]);
                        mma16816<MT>(o[nt][m], r, lo[kb][nt][0], lo[kb][nt][1]);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < P::CHUNKS / 2; ++j) {
                    uint32_t r[4];
                    ldmatrix4_trans(vs + P::chunk(row + (lane & 15), 2 * j + (lane >> 4)) * 16, r);
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t v[4] = {half2_of_e4m3(__byte_perm(r[2 * c], 0, 0x20)), half2_of_e4m3(__byte_perm(r[2 * c], 0, 0x31)),
                                               half2_of_e4m3(__byte_perm(r[2 * c + 1], 0, 0x20)), half2_of_e4m3(__byte_perm(r[2 * c + 1], 0, 0x31))};
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816<MT>(o[nt][2 * j + c], v, hi[kb][nt][0], hi[kb][nt][1]);
                            mma16816<MT>(o[nt][2 * j + c], v, lo[kb][nt][0], lo[kb][nt][1]);
                        }
                    }
                }
            }
        }

        if (flags & kTileLast) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    total[nt][i] = column_sum(total[nt][i]);
                    if (g8 == 0) {
                        s_top[warp][nt * 8 + 2 * t4 + i] = top[nt][i];
                        s_total[warp][nt * 8 + 2 * t4 + i] = total[nt][i];
                    }
                }
            __syncthreads();  // and every warp is done with the stage
            float* rows = reinterpret_cast<float*>(stage);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int head = nt * 8 + 2 * t4 + i;
                    float best = s_top[0][head];
#pragma unroll
                    for (int w = 1; w < kAttnWarps; ++w)
                        best = fmaxf(best, s_top[w][head]);
                    const float fix = exp2_fast(top[nt][i] - base_of(best)) * (1.0f / LIFT);
                    float* out = rows + (warp * P::HEADS + head) * P::OPITCH;
#pragma unroll
                    for (int m = 0; m < MTILES; ++m) {
                        out[m * 16 + (P::SMALL ? 2 * g8 : g8)] = o[nt][m][i] * fix;
                        out[m * 16 + (P::SMALL ? 2 * g8 + 1 : g8 + 8)] = o[nt][m][i + 2] * fix;
                    }
                }
            __syncthreads();
            write_part<P>(a, tile, run, first, began, rows, s_top, s_total);
            __syncthreads();  // the next copies go to this stage
        }
        feed.next();
    }
}

// ---------------------------------------------------------------------------
// The join of an item's parts, which lie in the slots of the blocks that the
// item's first block names; an item that one block had whole is written
// already.  A block takes `columns` (a power of two) of an item's groups of
// four elements, heads after each other; its threads take a column over every
// (threads / columns)-th part with a maximum and a sum of their own, all loads
// of four parts at once, and meet in a fixed tree in shared memory.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kJoinThreads, 4)  // 64 registers: a join fits beside attention blocks
k_attn_join(const AttnArgs a, const int columns)
{
    constexpr int AHEAD = 4;
    __shared__ float4 s_o[kJoinThreads];
    __shared__ float2 s_w[kJoinThreads];  // maximum and sum
    // The next kernel is not let in early here: blocks of the next attention that then filled the SMs beside waiting joins
    // lay unevenly, and the last of them ran as a second wave (93 MB of fp16 cache: 24.0 against 29 us a call).
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x;
    const int heads = a.kv_heads * a.group_blocks;
    const int slots = min(a.group, a.block_heads), fours = a.head_dim / 4;
    const int cuts = (slots * fours + columns - 1) / columns;
    const int item = blockIdx.x / cuts;
    const int2 blocks = a.blocks_of[item];
    const int c0 = blocks.x, c1 = blocks.y;
    if (c0 == c1)
        return;
    const int b = item / heads, hb = item - b * heads;
    const int parts = c1 - c0 + 1, groups = kJoinThreads / columns, group = tid / columns;
    const int x = (blockIdx.x - item * cuts) * columns + tid % columns;
    const int h = static_cast<int>(static_cast<uint32_t>(x) * a.fours_magic >> 32), e = (x - h * fours) * 4;
    const bool mine = h < heads_of(a, hb);
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float top = -INFINITY, total = 0.0f;
    for (int p0 = group; p0 < parts && mine; p0 += AHEAD * groups) {
        float4 v[AHEAD];
        float m[AHEAD], n[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int p = p0 + i * groups;
            m[i] = -INFINITY;
            n[i] = 0.0f;
            v[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (p < parts) {
                const float* part = a.part + slot_of(c0 + p, p == 0) * a.slot_floats;  // part 0 begins the item
                m[i] = part[slots * a.head_dim + h];
                n[i] = part[slots * (a.head_dim + 1) + h];
                v[i] = *reinterpret_cast<const float4*>(part + h * a.head_dim + e);
            }
        }
        float best = top;
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
            best = fmaxf(best, m[i]);
        const float base = best == -INFINITY ? 0.0f : best;
        float f = exp2f(top - base);
        top = best;
        total *= f;
        o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            f = exp2f(m[i] - base);
            total = fmaf(n[i], f, total);
            o = make_float4(fmaf(v[i].x, f, o.x), fmaf(v[i].y, f, o.y), fmaf(v[i].z, f, o.z), fmaf(v[i].w, f, o.w));
        }
    }
    for (int w = groups / 2; w > 0; w >>= 1) {
        if (group < 2 * w) {
            s_o[tid] = o;
            s_w[tid] = make_float2(top, total);
        }
        __syncthreads();
        if (group < w) {
            const float4 v = s_o[tid + w * columns];
            const float2 y = s_w[tid + w * columns];
            const float best = fmaxf(top, y.x), base = best == -INFINITY ? 0.0f : best;
            const float f = exp2f(top - base), g = exp2f(y.x - base);
            top = best;
            total = total * f + y.y * g;
            o = make_float4(o.x * f + v.x * g, o.y * f + v.y * g, o.z * f + v.z * g, o.w * f + v.w * g);
        }
        __syncthreads();
    }
    if (group == 0 && mine) {
        const uint64_t row = out_row(a, b, hb, h);
        store_four(reinterpret_cast<T*>(a.out) + row * a.head_dim + e, o, out_scale(a, total));
        if (e == 0 && a.lse != nullptr)
            a.lse[row] = lse_of(top, total);
    }
}

// Launches shape P's kernel, and then the join.
template <typename P>
cudaError_t launch_shape(void (*kernel)(AttnArgs), const AttnArgs& a, int most, int sms, cudaStream_t s)
{
    int per_sm = P::BLOCKS;
    const uint64_t items = static_cast<uint64_t>(a.batch) * a.kv_heads * a.group_blocks;
    // Few items: a third block an SM adds more to the join than it takes from the loads, unless the items are long.  With
    // two and three blocks, bf16 heads of 128: 17 MB in one item 10.9 and 14.2 us, in 8 11.3 and 12.7, in 16 11.2 and 12.7;
    // 67 MB in one 17.9 and 19.2, in 8 17.8 and 18.2, in 16 18.0 and 18.1; 134 MB of fp16 heads of 64 in 8 26.8 and 26.0, in
    // 16 26.7 and 26.0.  The lengths, which would tell more than the items, are not on the host.
    if (items <= 8 && per_sm > 2)
        per_sm = 2;
    const int blocks = most < sms * per_sm ? most : sms * per_sm;
    // The join's threads of a column: an eighth of the parts that an item has if all are alike, 32 at most, and two at
    // least, for one sequence may be much longer than the others (four cost 2 us more on 511 MB in 256 rows).
    int groups = 2;
    while (groups < 32 && 8ull * groups * items <= static_cast<uint64_t>(blocks))
        groups *= 2;
    const int columns = kJoinThreads / groups, slots = a.group < a.block_heads ? a.group : a.block_heads;
    const uint64_t joins = items * ((slots * (a.head_dim / 4) + columns - 1) / columns);
    if (joins > static_cast<uint64_t>(INT_MAX))
        return cudaErrorInvalidConfiguration;
    // The kernel's shared memory limit is raised once a device (0.4 us of a call's 7).  A context that was reset since has
    // lost it: its launch fails, and is made again with the limit raised.
    static std::atomic<uint64_t> raised{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    const bool before = (raised.load(std::memory_order_relaxed) & bit) != 0;
    const auto raise = [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, P::SMEM); };
    if (e == cudaSuccess && !before)
        e = raise();
    if (e == cudaSuccess)
        e = launch_k(kernel, dim3(blocks), dim3(kAttnThreads), P::SMEM, s, a);
    if (e == cudaErrorInvalidValue && before) {
        cudaGetLastError();
        e = raise();
        if (e == cudaSuccess)
            e = launch_k(kernel, dim3(blocks), dim3(kAttnThreads), P::SMEM, s, a);
    }
    if (e != cudaSuccess)
        return e;
    raised.fetch_or(bit, std::memory_order_relaxed);
    return launch_k(k_attn_join<typename P::T>, dim3(static_cast<unsigned>(joins)), dim3(kJoinThreads), 0, s, a, columns);
}

template <typename T, typename CT, int DIM, int HEADS>
cudaError_t launch_heads(const AttnArgs& a, int most, int sms, cudaStream_t s)
{
    using P = AttnShape<T, CT, DIM, HEADS>;
    if constexpr (P::WIDE)
        return launch_shape<P>(k_attn_fma<P>, a, most, sms, s);
    else
        return launch_shape<P>(k_attn_mma<P>, a, most, sms, s);
}

template <typename T, typename CT, int DIM>
cudaError_t launch_dim(const AttnArgs& a, int most, int sms, cudaStream_t s)
{
    if constexpr (sizeof(CT) == 4)
        return a.group <= 2 ? launch_heads<T, CT, DIM, 2>(a, most, sms, s) : launch_heads<T, CT, DIM, 8>(a, most, sms, s);
    else
        return a.group <= 8 ? launch_heads<T, CT, DIM, 8>(a, most, sms, s) : launch_heads<T, CT, DIM, 16>(a, most, sms, s);
}

template <typename T, typename CT>
cudaError_t launch_attention(const AttnArgs& a, int most, int sms, cudaStream_t s)
{
    return a.head_dim <= 64    ? launch_dim<T, CT, 64>(a, most, sms, s)
           : a.head_dim <= 96  ? launch_dim<T, CT, 96>(a, most, sms, s)
           : a.head_dim <= 128 ? launch_dim<T, CT, 128>(a, most, sms, s)
           : a.head_dim <= 192 ? launch_dim<T, CT, 192>(a, most, sms, s)
                               : launch_dim<T, CT, 256>(a, most, sms, s);
}

}  // namespace ar
