// ar_attn.cuh -- attention of one new token of each sequence over a paged
// key-value cache.
//
// Work split.  An item is one sequence, one key-value head and up to 16 of its
// query heads; its tokens are cut into tiles.  All items' tiles, in the order
// sequence, head, token, form one line, of which each block takes an equal
// run: blocks finish together whatever the lengths, one long sequence fills
// the GPU as well as many short ones, and the host needs no lengths.  A block
// finds its run by one scan over the lengths.  Rows whose tiles fell to more
// than one block leave a partial sum, maximum and weight in two slots per
// block, which k_attn_join adds up in block order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <type_traits>

#include "ar_cache.h"
#include "ar_kernels.cuh"
#include "ar_launch_k.cuh"

namespace ar {

constexpr int kAttnThreads = 128;
constexpr int kAttnWarps = kAttnThreads / 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 16-byte asynchronous copy into shared memory; `read` == false writes zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool read)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(read ? 16 : 0) : "memory");
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

// The run of tiles of block `c` of `blocks`: the first total % blocks blocks take one more.
struct Run {
    long long lo;
    long long n;
};
__device__ __forceinline__ Run run_of(long long total, int blocks, int c)
{
    const long long q = total / blocks, r = total % blocks;
    return {c * q + min(static_cast<long long>(c), r), q + (c < r)};
}
// The block whose run has tile x.
__device__ __forceinline__ int block_of(long long total, int blocks, long long x)
{
    const long long q = total / blocks, r = total % blocks, edge = r * (q + 1);
    return static_cast<int>(x < edge ? x / (q + 1) : r + (x - edge) / q);
}

// Where a block is on the line.
struct Cursor {
    int b, hb, tile;  // sequence, head and group block, tile of the item
    int next_length;  // of sequence b + 1, loaded when b began
    Span s;
    __device__ void fetch_next(const AttnArgs& a) { next_length = b + 1 < a.batch ? a.lengths[b + 1] : 0; }
    template <int TILE>
    __device__ void advance(const AttnArgs& a, int heads)
    {
        if (++tile < s.tiles)
            return;
        tile = 0;
        if (++hb < heads)
            return;
        hb = 0;
        ++b;
        s = span_of_length<TILE>(a, next_length);
        fetch_next(a);
    }
};

// Finds the block's run and its first tile.  All threads; contains barriers.
template <int TILE>
__device__ Run find_run(const AttnArgs& a, int heads, Cursor& cur)
{
    __shared__ int s_warp[kAttnWarps];
    __shared__ int s_b;
    __shared__ long long s_before;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // Tiles of the sequences [base, base + kAttnThreads), scanned: this thread's own are [before, before + mine).
    int mine = 0, before = 0, chunk = 0;
    const auto scan = [&](int base) {
        mine = base + tid < a.batch ? span_of<TILE>(a, base + tid).tiles : 0;
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(~0u, incl, o);
            incl += lane >= o ? up : 0;
        }
        if (lane == 31)
            s_warp[warp] = incl;
        __syncthreads();
        before = incl - mine;
        chunk = 0;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            before += w < warp ? s_warp[w] : 0;
            chunk += s_warp[w];
        }
        __syncthreads();
    };
    long long tiles = 0;
    for (int base = 0; base < a.batch; base += kAttnThreads) {
        scan(base);
        tiles += chunk;
    }
    const Run run = run_of(tiles * heads, gridDim.x, blockIdx.x);
    if (run.n == 0)
        return run;
    const long long x = run.lo / heads;  // sequence b takes [heads * P, heads * (P + tiles of b)) of the line
    long long passed = 0;
    for (int base = 0; base < a.batch; base += kAttnThreads) {
        if (a.batch > kAttnThreads)
            scan(base);
        if (x < passed + chunk) {
            const long long p = passed + before;
            if (p <= x && x < p + mine) {
                s_b = base + tid;
                s_before = p;
            }
            break;
        }
        passed += chunk;
    }
    __syncthreads();
    cur.b = s_b;
    cur.s = span_of<TILE>(a, cur.b);
    const long long in = run.lo - s_before * heads;
    cur.hb = static_cast<int>(in / cur.s.tiles);
    cur.tile = static_cast<int>(in % cur.s.tiles);
    cur.fetch_next(a);
    return run;
}

// One tile in flight: who it belongs to, and each token's offset in the cache (-1: left out).
enum { kTileFirst = 1, kTileLast = 2, kTileBegins = 4, kTileEnds = 8 };  // of the block's part; of the item
template <int TILE>
struct TileInfo {
    long long offset[TILE];
    int b, hb, flags, pad;
};

// Fills `info` for the cursor's tile, `t` of the run's `n`.
template <int TILE>
__device__ __forceinline__ void describe(const AttnArgs& a, const Cursor& cur, long long t, long long n, TileInfo<TILE>& info)
{
    const int tid = threadIdx.x;
    if (tid < TILE) {
        const int token = (cur.s.tile0 + cur.tile) * TILE + tid;
        long long off = -1;
        if (token >= cur.s.start && token < cur.s.end) {
            const uint32_t column = static_cast<uint32_t>(static_cast<uint64_t>(token) * a.page_magic >> a.page_shift);
            const int page = a.table[static_cast<uint64_t>(cur.b) * a.table_stride + column];
            if (page >= 0 && page < a.pages)
                off = static_cast<long long>(static_cast<uint64_t>(page) * a.page_stride +
                                             static_cast<uint64_t>(token - static_cast<int>(column) * a.page_size) * a.token_stride +
                                             static_cast<uint64_t>(cur.hb / a.group_blocks) * a.head_stride);
        }
        info.offset[tid] = off;
    }
    if (tid == 0) {
        const bool begins = cur.tile == 0, ends = cur.tile + 1 == cur.s.tiles;
        info.b = cur.b;
        info.hb = cur.hb;
        info.flags = (begins || t == 0 ? kTileFirst : 0) | (ends || t + 1 == n ? kTileLast : 0) |
                     (begins ? kTileBegins : 0) | (ends ? kTileEnds : 0);
    }
}

// Row of the output of head `i` of the item's group block, and how many heads the block has.
__device__ __forceinline__ uint64_t out_row(const AttnArgs& a, int b, int hb, int i)
{
    const int h = hb / a.group_blocks, gb = hb - h * a.group_blocks;
    return (static_cast<uint64_t>(b) * a.kv_heads + h) * a.group + gb * kAttnMaxHeads + i;
}
__device__ __forceinline__ int heads_of(const AttnArgs& a, int hb)
{
    return min(a.group - (hb % a.group_blocks) * kAttnMaxHeads, kAttnMaxHeads);
}

// A score in the exponent's base 2, of a dot product times scale2.
__device__ __forceinline__ float score2(const AttnArgs& a, float s)
{
    return a.softcap > 0.0f ? a.softcap2 * tanhf(s) : s;
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

template <typename CT>
__device__ __forceinline__ float cached_to_f(CT v)
{
    if constexpr (sizeof(CT) == 1)
        return static_cast<float>(v);
    else
        return Lanes<CT>::to_f(v);
}

// ---------------------------------------------------------------------------
// The plain-arithmetic kernel: fp32 multiply-adds.  Tiles come through a ring
// of asynchronous copies; a warp's lanes take one token each and the warps
// share the heads for the scores, the threads take one element of the head
// each for the weighted values, so no sum ever crosses a thread.
// ---------------------------------------------------------------------------
template <typename T, typename CT, int DIM, int HEADS>
struct PlainShape {
    static constexpr int TILE = 32;
    static constexpr int STAGES = 3;
    static constexpr int VE = 16 / sizeof(CT);
    static constexpr int CHUNKS = DIM / VE;
    static constexpr int PITCH = DIM * sizeof(CT) + 16;  // an odd number of 16-byte words: lanes meet no bank twice
    static constexpr int TILE_BYTES = TILE * PITCH;
    static constexpr int ITEM = STAGES * 2 * TILE_BYTES;
    static constexpr int SMEM = ITEM + HEADS * DIM * 4 + TILE * HEADS * 4;
    static constexpr int BLOCKS = SMEM + 2048 + kSmemReservedPerBlock <= kSmemPerSM / 2 ? 2 : 1;
    // Threads over the head's elements, and over groups of heads where the elements leave some over.
    static constexpr int DT = DIM == 192 ? 96 : (DIM < 128 ? DIM : 128);
    static constexpr int HS = 128 / DT;
    static constexpr int DPT = DIM / DT;
    static constexpr int NH = (HEADS + HS - 1) / HS;
    static constexpr int HPW = (HEADS + kAttnWarps - 1) / kAttnWarps;
};

template <typename T, typename CT, int DIM, int HEADS>
__global__ void __launch_bounds__(kAttnThreads, PlainShape<T, CT, DIM, HEADS>::BLOCKS)
k_attn_plain(const AttnArgs a)
{
    using P = PlainShape<T, CT, DIM, HEADS>;
    constexpr int TILE = P::TILE, RING = P::STAGES + 1;
    extern __shared__ __align__(16) char smem[];
    __shared__ TileInfo<TILE> s_info[RING];
    __shared__ float s_top[HEADS], s_total[HEADS], s_fix[HEADS];
    float* s_q = reinterpret_cast<float*>(smem + P::ITEM);  // [HEADS][DIM]
    float* s_p = s_q + HEADS * DIM;                         // [TILE][HEADS]
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int heads = a.kv_heads * a.group_blocks;
    const int chunks = a.head_dim / P::VE;

    Cursor cur;
    const Run run = find_run<TILE>(a, heads, cur);
    if (run.n == 0)
        return;

    long long described = 0;
    const auto next_info = [&] {
        if (described < run.n) {
            describe<TILE>(a, cur, described, run.n, s_info[described % RING]);
            cur.advance<TILE>(a, heads);
        }
        ++described;
    };
    const auto issue = [&](long long t) {
        if (t < run.n) {
            const TileInfo<TILE>& info = s_info[t % RING];
            char* stage = smem + (t % P::STAGES) * 2 * P::TILE_BYTES;
            for (int x = tid; x < TILE * P::CHUNKS; x += kAttnThreads) {
                const int row = x / P::CHUNKS, c = x - row * P::CHUNKS;
                if (c < chunks) {
                    const long long off = info.offset[row];
                    const uint32_t dst = smem_addr(stage + row * P::PITCH + c * 16);
                    const long long at = (off < 0 ? 0 : off) + c * 16;
                    cp_async16(dst, a.k + at, off >= 0);
                    cp_async16(dst + P::TILE_BYTES, a.v + at, off >= 0);
                }
            }
        }
        cp_async_commit();
    };
    for (int i = 0; i < P::STAGES; ++i)
        next_info();
    __syncthreads();
    for (int i = 0; i + 1 < P::STAGES; ++i)
        issue(i);

    const int d0 = tid % P::DT, hs = tid / P::DT;
    float o[P::NH][P::DPT];
    bool began = false;  // the block's part of the item holds its first tile
    for (long long t = 0; t < run.n; ++t) {
        cp_async_wait<P::STAGES - 2>();
        __syncthreads();
        issue(t + P::STAGES - 1);
        const TileInfo<TILE>& info = s_info[t % RING];
        const char* ks = smem + (t % P::STAGES) * 2 * P::TILE_BYTES;
        const char* vs = ks + P::TILE_BYTES;
        const int g = heads_of(a, info.hb);
        if (info.flags & kTileFirst) {
            began = info.flags & kTileBegins;
            const T* q = reinterpret_cast<const T*>(a.q + info.b * a.q_stride) +
                         (out_row(a, 0, info.hb, 0)) * a.head_dim;
            for (int x = tid; x < g * a.head_dim; x += kAttnThreads) {
                const int h = x / a.head_dim;
                s_q[h * DIM + x - h * a.head_dim] = Lanes<T>::to_f(q[x]);
            }
            if (tid < HEADS) {
                s_top[tid] = -INFINITY;
                s_total[tid] = 0.0f;
            }
#pragma unroll
            for (int h = 0; h < P::NH; ++h)
#pragma unroll
                for (int d = 0; d < P::DPT; ++d)
                    o[h][d] = 0.0f;
            __syncthreads();
        }
        // Scores: lane = token, heads over warps.
        {
            float dot[P::HPW];
#pragma unroll
            for (int i = 0; i < P::HPW; ++i)
                dot[i] = 0.0f;
            for (int c = 0; c < chunks; ++c) {
                const CT* kc = reinterpret_cast<const CT*>(ks + lane * P::PITCH + c * 16);
                float k[P::VE];
                const uint4 raw = *reinterpret_cast<const uint4*>(kc);
                const CT* e = reinterpret_cast<const CT*>(&raw);
#pragma unroll
                for (int l = 0; l < P::VE; ++l)
                    k[l] = cached_to_f(e[l]);
#pragma unroll
                for (int i = 0; i < P::HPW; ++i) {
                    const int h = warp + i * kAttnWarps;
                    if (h < g) {
                        const float* q = s_q + h * DIM + c * P::VE;
#pragma unroll
                        for (int l = 0; l < P::VE; ++l)
                            dot[i] = fmaf(q[l], k[l], dot[i]);
                    }
                }
            }
            const bool in = info.offset[lane] >= 0;
#pragma unroll
            for (int i = 0; i < P::HPW; ++i) {
                const int h = warp + i * kAttnWarps;
                if (h < g) {
                    const float x = in ? score2(a, dot[i] * a.scale2) : -INFINITY;
                    float top = x;
#pragma unroll
                    for (int w = 16; w > 0; w >>= 1)
                        top = fmaxf(top, __shfl_xor_sync(~0u, top, w));
                    const float old = s_top[h];
                    top = fmaxf(top, old);
                    const float base = top == -INFINITY ? 0.0f : top;
                    const float p = exp2f(x - base);
                    float sum = p;
#pragma unroll
                    for (int w = 16; w > 0; w >>= 1)
                        sum += __shfl_xor_sync(~0u, sum, w);
                    s_p[lane * HEADS + h] = p;
                    __syncwarp();
                    if (lane == 0) {
                        const float fix = exp2f(old - base);
                        s_fix[h] = fix;
                        s_total[h] = s_total[h] * fix + sum;
                        s_top[h] = top;
                    }
                }
            }
        }
        __syncthreads();
        // Weighted values: thread = element of the head.
        if (hs < P::HS) {
#pragma unroll
            for (int h = 0; h < P::NH; ++h) {
                const float fix = s_fix[min(hs * P::NH + h, HEADS - 1)];
#pragma unroll
                for (int d = 0; d < P::DPT; ++d)
                    o[h][d] = hs * P::NH + h < g ? o[h][d] * fix : 0.0f;
            }
#pragma unroll 4
            for (int j = 0; j < TILE; ++j) {
                float v[P::DPT];
#pragma unroll
                for (int d = 0; d < P::DPT; ++d)
                    v[d] = cached_to_f(reinterpret_cast<const CT*>(vs + j * P::PITCH)[d0 + d * P::DT]);
#pragma unroll
                for (int h = 0; h < P::NH; ++h) {
                    if (hs * P::NH + h < g) {
                        const float p = s_p[j * HEADS + hs * P::NH + h];
#pragma unroll
                        for (int d = 0; d < P::DPT; ++d)
                            o[h][d] = fmaf(p, v[d], o[h][d]);
                    }
                }
            }
        }
        if (info.flags & kTileLast) {
            const bool whole = began && (info.flags & kTileEnds);
            const int slots = min(a.group, kAttnMaxHeads);
            float* part = a.part + (2ull * blockIdx.x + (began ? 1 : 0)) * a.slot_floats;
#pragma unroll
            for (int h = 0; h < P::NH; ++h) {
                const int head = hs * P::NH + h;
                if (hs < P::HS && head < g) {
                    const uint64_t row = out_row(a, info.b, info.hb, head);
                    const float f = out_scale(a, s_total[head]);
#pragma unroll
                    for (int d = 0; d < P::DPT; ++d) {
                        const int e = d0 + d * P::DT;
                        if (e < a.head_dim) {
                            if (whole)
                                reinterpret_cast<T*>(a.out)[row * a.head_dim + e] = Lanes<T>::from_f(o[h][d] * f);
                            else
                                part[head * a.head_dim + e] = o[h][d];
                        }
                    }
                }
            }
            if (tid < g) {
                if (!whole) {
                    part[slots * a.head_dim + tid] = s_top[tid];
                    part[slots * (a.head_dim + 1) + tid] = s_total[tid];
                } else if (a.lse != nullptr) {
                    a.lse[out_row(a, info.b, info.hb, tid)] = lse_of(s_top[tid], s_total[tid]);
                }
            }
            __syncthreads();  // the next item's first tile writes s_top and s_total
        }
        next_info();
    }
}

// ---------------------------------------------------------------------------
// The matrix kernel, for 16-bit and 8-bit caches.  Scores are computed as
// K Q^T and values as V^T P^T: tokens, and then the head's elements, are the
// 16 rows of a matrix instruction and query heads its 8 columns, so that up to
// 8 heads fill it where rows of queries would leave half of it empty, and both
// operands from the cache come out of shared memory by ldmatrix as they lie
// there.  Each warp takes a quarter of a tile's tokens, through a ring of its
// own, with a maximum, a sum and an accumulator of its own: the four meet at the
// ends of the block's part of an item only, and between them no warp waits for
// another.  Weights enter the second product as a pair of 16-bit
// numbers, their rounding and what it leaves (17 bits and more together), which
// costs an instruction that the memory's pace hides.  8-bit elements become
// fp16 in registers, exactly; queries too large or small for fp16 are scaled
// by a power of two per head first.
// ---------------------------------------------------------------------------
template <typename T, typename CT, int DIM, int NT>
struct MmaShape {
    static constexpr bool SMALL = sizeof(CT) == 1;
    using MT = typename std::conditional<SMALL, __half, CT>::type;  // of the matrix instructions' operands
    static constexpr int TILE = attn_tile(sizeof(CT));
    static constexpr int TOKENS = TILE / kAttnWarps;  // a warp's tokens of a tile
    static constexpr int KB = TOKENS / 16;            // and their blocks of 16
    static constexpr int CHUNKS = DIM * sizeof(CT) / 16;
    static constexpr int QCHUNKS = DIM * sizeof(T) / 16;
    // 16-byte chunks of a row: permuted within 128 bytes by the row, or padded to an odd number; either way the eight
    // rows of an 8 x 8 matrix lie in different banks.
    static constexpr int PITCH = CHUNKS % 8 == 0 ? CHUNKS : CHUNKS | 1;
    static constexpr int QPITCH = QCHUNKS % 8 == 0 ? QCHUNKS : QCHUNKS | 1;
    static constexpr int HALF = TOKENS * PITCH * 16;  // a warp's keys of a stage, and its values
    static constexpr int QROWS = kAttnWarps * 2 * HALF;  // where a stage's queries begin
    static constexpr int STAGE = QROWS + 8 * NT * QPITCH * 16;
    static constexpr int INFO = kAttnWarps * (TOKENS * 8 + 16);
    static constexpr int OPITCH = DIM + 4;  // floats; the epilogue's rows, one per warp and head, lie in a used stage
    static_assert(kAttnWarps * 8 * NT * OPITCH * 4 <= STAGE, "the epilogue fits a stage");
    static constexpr int fits(int bytes)
    {
        const int n = (bytes - kSmemReservedPerBlock - 1024 - INFO) / (STAGE + INFO);
        return n < 5 ? n : 5;
    }
    // Blocks of an SM.  A tile of few bytes takes a warp longer than they take to come, so that more warps help: four
    // blocks of heads up to 64 elements (31.8 against 34.3 us with two on 93 MB of fp16 cache), three of 8-bit ones up to
    // 128 (93.5 against 98.6 us on 533 MB).  For 128 16-bit elements two blocks' deeper rings do better (93 against 98 us
    // on 511 MB).  Long heads leave room for two stages in one block only.
    static constexpr int WANT = NT == 1 && DIM <= 64 ? 4 : NT == 1 && DIM <= 128 && SMALL ? 3 : 2;
    static constexpr int BLOCKS = fits(kSmemPerSM / WANT) >= 2 ? WANT : 1;
    static constexpr int STAGES = fits(kSmemPerSM / BLOCKS);
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
template <int TOKENS>
struct WarpTile {
    long long offset[TOKENS];
    int b, hb, flags;
    uint32_t in;
};

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
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Maximum or sum over the eight lanes that hold the same column.
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

template <typename T, typename CT, int DIM, int NT>
__global__ void __launch_bounds__(kAttnThreads, MmaShape<T, CT, DIM, NT>::BLOCKS)
k_attn_mma(const AttnArgs a)
{
    using P = MmaShape<T, CT, DIM, NT>;
    using MT = typename P::MT;
    constexpr int TILE = P::TILE, TOKENS = P::TOKENS, RING = P::STAGES + 1, KB = P::KB, MTILES = DIM / 16, KSTEPS = DIM / 16;
    extern __shared__ __align__(128) char smem[];
    __shared__ __align__(16) WarpTile<TOKENS> s_tiles[kAttnWarps][RING];
    __shared__ float s_top[kAttnWarps][8 * NT], s_total[kAttnWarps][8 * NT];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, t4 = lane & 3;
    const int heads = a.kv_heads * a.group_blocks;
    const int chunks = a.head_dim * static_cast<int>(sizeof(CT)) / 16;
    const int qchunks = a.head_dim * static_cast<int>(sizeof(T)) / 16;

    Cursor cur;
    const Run run = find_run<TILE>(a, heads, cur);
    if (run.n == 0)
        return;
    const int n = static_cast<int>(min(run.n, static_cast<long long>(INT_MAX)));

    // The description of the cursor's tile, `t` of the run, in two steps: its pages' numbers are on their way between them.
    WarpTile<TOKENS>* const tiles = s_tiles[warp];
    int page = -1, slot = 0;
    const auto look_up = [&] {
        const int token = (cur.s.tile0 + cur.tile) * TILE + warp * TOKENS + lane;
        page = -1;
        if (lane < TOKENS && token >= cur.s.start && token < cur.s.end) {
            const uint32_t column = static_cast<uint32_t>(static_cast<uint64_t>(token) * a.page_magic >> a.page_shift);
            slot = token - static_cast<int>(column) * a.page_size;
            page = a.table[static_cast<uint64_t>(cur.b) * a.table_stride + column];
        }
    };
    const auto describe_tile = [&](int t, WarpTile<TOKENS>& tile) {
        const bool in = page >= 0 && page < a.pages;
        const uint32_t mask = __ballot_sync(~0u, in);
        if (lane < TOKENS)
            tile.offset[lane] = in ? static_cast<long long>(static_cast<uint64_t>(page) * a.page_stride +
                                                            static_cast<uint64_t>(slot) * a.token_stride +
                                                            static_cast<uint64_t>(cur.hb / a.group_blocks) * a.head_stride)
                                   : 0;
        if (lane == 0) {
            const bool begins = cur.tile == 0, ends = cur.tile + 1 == cur.s.tiles;
            tile.b = cur.b;
            tile.hb = cur.hb;
            tile.flags = (begins || t == 0 ? kTileFirst : 0) | (ends || t + 1 == n ? kTileLast : 0) |
                         (begins ? kTileBegins : 0) | (ends ? kTileEnds : 0);
            tile.in = mask;
        }
        cur.advance<TILE>(a, heads);
    };
    // The warp's copies of a described tile.  Chunks beyond the head's elements and tokens that are left out become zeros.
    const auto issue = [&](const WarpTile<TOKENS>& tile, int stage) {
        const uint32_t base = smem_addr(smem + stage * P::STAGE);
        const uint32_t ks = base + warp * 2 * P::HALF;
        const uint32_t in = tile.in;
#pragma unroll
        for (int i = 0; i < TOKENS * P::CHUNKS / 32; ++i) {
            int row, c;
            if constexpr (32 % P::CHUNKS == 0) {
                row = i * (32 / P::CHUNKS) + lane / P::CHUNKS;
                c = lane % P::CHUNKS;
            } else {
                row = (lane + i * 32) / P::CHUNKS;
                c = lane + i * 32 - row * P::CHUNKS;
            }
            const bool read = (in >> row & 1) != 0 && c < chunks;
            const long long at = tile.offset[row] + (c < chunks ? c * 16 : 0);
            const uint32_t dst = ks + P::chunk(row, c) * 16;
            cp_async16(dst, a.k + at, read);
            cp_async16(dst + P::HALF, a.v + at, read);
        }
        if (tile.flags & kTileFirst) {
            const int g = heads_of(a, tile.hb);
            const char* q = a.q + tile.b * a.q_stride + out_row(a, 0, tile.hb, 0) * a.head_dim * sizeof(T);
            for (int x = tid; x < 8 * NT * P::QCHUNKS; x += kAttnThreads) {
                const int row = x / P::QCHUNKS, c = x - row * P::QCHUNKS;
                const bool read = row < g && c < qchunks;
                cp_async16(base + P::QROWS + P::qchunk(row, c) * 16,
                           q + (read ? static_cast<size_t>(row) * a.head_dim * sizeof(T) + c * 16 : 0), read);
            }
        }
    };

    int described = 0, ring_w = 0;  // the next tile to describe, and its slot of the ring
#pragma unroll 1
    for (; described < P::STAGES && described < n; ++described) {
        look_up();
        describe_tile(described, tiles[ring_w]);
        ++ring_w;
    }
    __syncwarp();
#pragma unroll 1
    for (int i = 0; i + 1 < P::STAGES; ++i) {
        if (i < n)
            issue(tiles[i], i);
        cp_async_commit();
    }

    uint32_t qf[NT][KSTEPS][2];
    float o[NT][MTILES][4], top[NT][2], total[NT][2], qscale[NT][2];
    bool began = false;
    int ring_r = 0, ring_i = P::STAGES - 1, stage_r = 0, stage_w = P::STAGES - 1;
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
        cp_async_wait<P::STAGES - 2>();
        __syncwarp();
        if (t + P::STAGES - 1 < n)
            issue(tiles[ring_i], stage_w);
        cp_async_commit();
        if (described < n)
            look_up();
        const WarpTile<TOKENS>& tile = tiles[ring_r];
        const int flags = tile.flags;
        char* stage = smem + stage_r * P::STAGE;
        const uint32_t ks = smem_addr(stage) + warp * 2 * P::HALF, vs = ks + P::HALF, qs = smem_addr(stage) + P::QROWS;
        if (flags & kTileFirst)
            __syncthreads();  // the queries are the block's
        if (flags & kTileFirst) {
            began = flags & kTileBegins;
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
                    int e = 0;
                    if constexpr (!std::is_same<T, __half>::value) {
                        most = fmaxf(most, __shfl_xor_sync(~0u, most, 1));
                        most = fmaxf(most, __shfl_xor_sync(~0u, most, 2));
                        e = min(max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -126), 126);
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
                        qscale[nt][i] = ldexpf(a.scale2, eh);
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
                        s[kb][nt][i] = a.softcap2 * tanhf(s[kb][nt][i]);
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
                    // A maximum of minus infinity stands still here: 0 in its place keeps the difference defined.
                    const float fix = exp2_fast(top[nt][i] - (base[i] == -INFINITY ? 0.0f : base[i]));
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
                base[i] = base[i] == -INFINITY ? 0.0f : base[i];
#pragma unroll
            for (int kb = 0; kb < KB; ++kb) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float p0 = exp2_fast(s[kb][nt][2 * r] - base[0]);
                    const float p1 = exp2_fast(s[kb][nt][2 * r + 1] - base[1]);
                    total[nt][0] += p0;
                    total[nt][1] += p1;
                    const uint32_t h = Lanes<MT>::word(p0, p1);
                    const float2 back = Lanes<MT>::two(h);
                    hi[kb][nt][r] = transposed(h);
                    lo[kb][nt][r] = transposed(Lanes<MT>::word(p0 - back.x, p1 - back.y));
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
                    const float fix = exp2_fast(top[nt][i] - (best == -INFINITY ? 0.0f : best));
                    float* out = rows + (warp * 8 * NT + head) * P::OPITCH;
#pragma unroll
                    for (int m = 0; m < MTILES; ++m) {
                        out[m * 16 + (P::SMALL ? 2 * g8 : g8)] = o[nt][m][i] * fix;
                        out[m * 16 + (P::SMALL ? 2 * g8 + 1 : g8 + 8)] = o[nt][m][i + 2] * fix;
                    }
                }
            __syncthreads();
            const bool whole = began && (flags & kTileEnds);
            const int g = heads_of(a, tile.hb), fours = a.head_dim / 4;
            const int slots = min(a.group, kAttnMaxHeads);
            float* part = a.part + (2ull * blockIdx.x + (began ? 1 : 0)) * a.slot_floats;
            for (int x = tid; x < g * fours; x += kAttnThreads) {
                const int head = x / fours, d = (x - head * fours) * 4;
                float best = s_top[0][head], sum = 0.0f;
#pragma unroll
                for (int w = 1; w < kAttnWarps; ++w)
                    best = fmaxf(best, s_top[w][head]);
                const float base = best == -INFINITY ? 0.0f : best;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kAttnWarps; ++w) {
                    sum += s_total[w][head] * exp2_fast(s_top[w][head] - base);
                    const float4 y = *reinterpret_cast<const float4*>(rows + (w * 8 * NT + head) * P::OPITCH + d);
                    v.x += y.x;
                    v.y += y.y;
                    v.z += y.z;
                    v.w += y.w;
                }
                if (whole) {
                    const uint64_t row = out_row(a, tile.b, tile.hb, head);
                    const float f = out_scale(a, sum);
                    *reinterpret_cast<uint2*>(a.out + (row * a.head_dim + d) * sizeof(T)) =
                        make_uint2(Lanes<T>::word(v.x * f, v.y * f), Lanes<T>::word(v.z * f, v.w * f));
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
            __syncthreads();  // the next copies go to this stage
        }
        if (described < n) {
            describe_tile(described, tiles[ring_w]);
            ++described;
            ring_w = ring_w + 1 == RING ? 0 : ring_w + 1;
        }
        ring_r = ring_r + 1 == RING ? 0 : ring_r + 1;
        ring_i = ring_i + 1 == RING ? 0 : ring_i + 1;
        stage_r = stage_r + 1 == P::STAGES ? 0 : stage_r + 1;
        stage_w = stage_w + 1 == P::STAGES ? 0 : stage_w + 1;
    }
}

// ---------------------------------------------------------------------------
// The join of an item's parts.  It derives the blocks that hold parts from the
// same lengths and the same split; an item that one block had whole is written
// already.  A block takes `columns` (a power of two) of an item's groups of
// four elements, heads after each other; its threads take a column over every
// (threads / columns)-th part with a maximum and a sum of their own, all loads
// of eight parts at once, and meet in a fixed tree in shared memory.
// ---------------------------------------------------------------------------
constexpr int kJoinThreads = 256;

template <typename T, int TILE>
__global__ void __launch_bounds__(kJoinThreads)
k_attn_join(const AttnArgs a, const int blocks, const int columns)
{
    constexpr int WARPS = kJoinThreads / 32, AHEAD = 8;
    __shared__ long long s_sum[2][WARPS];
    __shared__ float4 s_o[kJoinThreads];
    __shared__ float2 s_w[kJoinThreads];  // maximum and sum
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int heads = a.kv_heads * a.group_blocks;
    const int slots = min(a.group, kAttnMaxHeads), fours = a.head_dim / 4;
    const int cuts = (slots * fours + columns - 1) / columns;
    const int item = blockIdx.x / cuts;
    const int b = item / heads, hb = item - b * heads;

    long long before = 0, all = 0;
    for (int s = tid; s < a.batch; s += kJoinThreads) {
        const int n = span_of<TILE>(a, s).tiles;
        all += n;
        before += s < b ? n : 0;
    }
    const int tiles = span_of<TILE>(a, b).tiles;
    if (a.batch > 1) {
#pragma unroll
        for (int w = 16; w > 0; w >>= 1) {
            all += __shfl_xor_sync(~0u, all, w);
            before += __shfl_xor_sync(~0u, before, w);
        }
        if (lane == 0) {
            s_sum[0][warp] = all;
            s_sum[1][warp] = before;
        }
        __syncthreads();
        all = before = 0;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            all += s_sum[0][w];
            before += s_sum[1][w];
        }
    } else {
        all = tiles;
    }
    const long long lo = before * heads + static_cast<long long>(hb) * tiles;
    const int c0 = block_of(all * heads, blocks, lo), c1 = block_of(all * heads, blocks, lo + tiles - 1);
    if (c0 == c1)
        return;
    const int parts = c1 - c0 + 1, groups = kJoinThreads / columns, group = tid / columns;
    const int x = (blockIdx.x - item * cuts) * columns + tid % columns;
    const int h = x / fours, e = (x - h * fours) * 4;
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
                // Part 0 lies in its block's slot 1 (it begins the item), the others in their blocks' slots 0.
                const float* part = a.part + (2ull * (c0 + p) + (p == 0 ? 1 : 0)) * a.slot_floats;
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
        const float f = out_scale(a, total);
        T* out = reinterpret_cast<T*>(a.out) + row * a.head_dim + e;
        if constexpr (sizeof(T) == 4)
            *reinterpret_cast<float4*>(out) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
        else
            *reinterpret_cast<uint2*>(out) = make_uint2(Lanes<T>::word(o.x * f, o.y * f), Lanes<T>::word(o.z * f, o.w * f));
        if (e == 0 && a.lse != nullptr)
            a.lse[row] = lse_of(top, total);
    }
}

// Launches `kernel`, `per_sm` blocks of which fit an SM, and then the join.
template <typename T, int TILE, typename Kernel>
cudaError_t launch_tiles(Kernel kernel, const AttnArgs& a, int most, int sms, int per_sm, size_t smem, cudaStream_t s)
{
    // The join's threads of a column: a quarter of the parts an item has if all are alike, four at least (one sequence
    // may be much longer than the others), 32 at most.
    const int blocks = most < sms * per_sm ? most : sms * per_sm;
    const uint64_t items = static_cast<uint64_t>(a.batch) * a.kv_heads * a.group_blocks;
    int groups = 4;
    while (groups < 32 && 8ull * groups * items <= static_cast<uint64_t>(blocks))
        groups *= 2;
    const int columns = kJoinThreads / groups, slots = a.group < kAttnMaxHeads ? a.group : kAttnMaxHeads;
    const uint64_t joins = items * ((slots * (a.head_dim / 4) + columns - 1) / columns);
    if (joins > static_cast<uint64_t>(INT_MAX))
        return cudaErrorInvalidConfiguration;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess)
        return e;
    e = launch_k(kernel, dim3(blocks), dim3(kAttnThreads), smem, s, a);
    if (e != cudaSuccess)
        return e;
    return launch_k(k_attn_join<T, TILE>, dim3(static_cast<unsigned>(joins)), dim3(kJoinThreads), 0, s, a, blocks, columns);
}

template <typename T, typename CT, int DIM, int HEADS>
cudaError_t launch_heads(const AttnArgs& a, int most, int sms, cudaStream_t s)
{
    constexpr int TILE = attn_tile(sizeof(CT));
    if constexpr (sizeof(CT) == 4) {
        using P = PlainShape<T, CT, DIM, HEADS>;
        return launch_tiles<T, TILE>(k_attn_plain<T, CT, DIM, HEADS>, a, most, sms, P::BLOCKS, P::SMEM, s);
    } else {
        using P = MmaShape<T, CT, DIM, HEADS / 8>;
        return launch_tiles<T, TILE>(k_attn_mma<T, CT, DIM, HEADS / 8>, a, most, sms, P::BLOCKS, P::SMEM, s);
    }
}

template <typename T, typename CT, int DIM>
cudaError_t launch_dim(const AttnArgs& a, int most, int sms, cudaStream_t s)
{
    if constexpr (sizeof(CT) == 4) {
        if (a.group <= 2)
            return launch_heads<T, CT, DIM, 2>(a, most, sms, s);
    }
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
