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
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b)
{
    Span s;
    s.end = min(max(a.lengths[b], 0), a.capacity);
    s.start = a.window > 0 ? max(s.end - a.window, 0) : 0;
    s.tile0 = s.start / TILE;
    s.tiles = max((s.end + TILE - 1) / TILE - s.tile0, 1);
    return s;
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
    Span s;
    template <int TILE>
    __device__ void advance(const AttnArgs& a, int heads)
    {
        if (++tile < s.tiles)
            return;
        tile = 0;
        if (++hb < heads)
            return;
        hb = 0;
        if (++b < a.batch)
            s = span_of<TILE>(a, b);
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
    return run;
}

// One tile in flight: who it belongs to, and each token's offset in the cache (-1: left out).
enum { kTileFirst = 1, kTileLast = 2, kTileBegins = 4, kTileEnds = 8 };  // of the block's part; of the item
template <int TILE>
struct TileInfo {
    long long offset[TILE];
    int b, hb, flags, pad;
};

// Fills `info` for the cursor's tile, `t` of the run's `n`.  Threads of [0, TILE).
template <int TILE>
__device__ __forceinline__ void describe(const AttnArgs& a, const Cursor& cur, long long t, long long n, TileInfo<TILE>& info)
{
    const int tid = threadIdx.x;
    if (tid < TILE) {
        const int token = (cur.s.tile0 + cur.tile) * TILE + tid;
        long long off = -1;
        if (token >= cur.s.start && token < cur.s.end) {
            const int column = token / a.page_size;
            const int page = a.table[static_cast<uint64_t>(cur.b) * a.table_stride + column];
            if (page >= 0 && page < a.pages)
                off = static_cast<long long>(static_cast<uint64_t>(page) * a.page_stride +
                                             static_cast<uint64_t>(token - column * a.page_size) * a.token_stride +
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

// A score in the exponent's base 2.
__device__ __forceinline__ float score2(const AttnArgs& a, float dot)
{
    const float s = dot * a.scale;
    return (a.softcap > 0.0f ? a.softcap * tanhf(s / a.softcap) : s) * kLog2e;
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
    // Threads over the head's elements, and over groups of heads where the elements leave some over.
    static constexpr int DT = DIM == 192 ? 96 : (DIM < 128 ? DIM : 128);
    static constexpr int HS = 128 / DT;
    static constexpr int DPT = DIM / DT;
    static constexpr int NH = (HEADS + HS - 1) / HS;
    static constexpr int HPW = (HEADS + kAttnWarps - 1) / kAttnWarps;
};

template <typename T, typename CT, int DIM, int HEADS>
__global__ void __launch_bounds__(kAttnThreads, 2)
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
                    const float x = in ? score2(a, dot[i]) : -INFINITY;
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
// The join of an item's parts: one block per item and head.  It derives the
// blocks that hold parts from the same lengths and the same split; an item
// that one block had whole is written already.  Warps take every fourth part,
// lanes the row's elements; the warps' sums are added in order.
// ---------------------------------------------------------------------------
template <typename T, int TILE>
__global__ void __launch_bounds__(kAttnThreads)
k_attn_join(const AttnArgs a, const int blocks)
{
    __shared__ long long s_sum[2][kAttnWarps];
    __shared__ float s_top[kAttnWarps], s_total[kAttnWarps];
    __shared__ float s_o[kAttnWarps][kAttnMaxDim];
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int heads = a.kv_heads * a.group_blocks;
    const int slots = min(a.group, kAttnMaxHeads);
    const int i = blockIdx.x % slots;
    const int item = blockIdx.x / slots;
    const int b = item / heads, hb = item - b * heads;

    long long before = 0, all = 0;
    for (int s = tid; s < a.batch; s += kAttnThreads) {
        const int n = span_of<TILE>(a, s).tiles;
        all += n;
        before += s < b ? n : 0;
    }
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
    for (int w = 0; w < kAttnWarps; ++w) {
        all += s_sum[0][w];
        before += s_sum[1][w];
    }
    const int tiles = span_of<TILE>(a, b).tiles;
    const long long lo = before * heads + static_cast<long long>(hb) * tiles;
    const int c0 = block_of(all * heads, blocks, lo), c1 = block_of(all * heads, blocks, lo + tiles - 1);
    if (c0 == c1 || i >= heads_of(a, hb))
        return;

    constexpr int DPL = kAttnMaxDim / 32;
    float o[DPL], top = -INFINITY, total = 0.0f;
#pragma unroll
    for (int d = 0; d < DPL; ++d)
        o[d] = 0.0f;
    for (int c = c0 + warp; c <= c1; c += kAttnWarps) {
        const float* part = a.part + (2ull * c + (c == c0 ? 1 : 0)) * a.slot_floats;
        const float m = part[slots * a.head_dim + i], n = part[slots * (a.head_dim + 1) + i];
        const float next = fmaxf(top, m), base = next == -INFINITY ? 0.0f : next;
        const float fix = exp2f(top - base), f = exp2f(m - base);
        total = total * fix + n * f;
        top = next;
#pragma unroll
        for (int d = 0; d < DPL; ++d) {
            const int e = lane + 32 * d;
            if (e < a.head_dim)
                o[d] = o[d] * fix + part[i * a.head_dim + e] * f;
        }
    }
#pragma unroll
    for (int d = 0; d < DPL; ++d)
        s_o[warp][lane + 32 * d] = o[d];
    if (lane == 0) {
        s_top[warp] = top;
        s_total[warp] = total;
    }
    __syncthreads();
    float best = -INFINITY;
    for (int w = 0; w < kAttnWarps; ++w)
        best = fmaxf(best, s_top[w]);
    const float base = best == -INFINITY ? 0.0f : best;
    float f[kAttnWarps], sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        f[w] = exp2f(s_top[w] - base);
        sum += s_total[w] * f[w];
    }
    const uint64_t row = out_row(a, b, hb, i);
    const float scale = out_scale(a, sum);
    for (int e = tid; e < a.head_dim; e += kAttnThreads) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w)
            v += s_o[w][e] * f[w];
        reinterpret_cast<T*>(a.out)[row * a.head_dim + e] = Lanes<T>::from_f(v * scale);
    }
    if (tid == 0 && a.lse != nullptr)
        a.lse[row] = lse_of(best, sum);
}

template <typename Kernel>
cudaError_t launch_tiles(Kernel kernel, const AttnArgs& a, int blocks, size_t smem, cudaStream_t s)
{
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    return e != cudaSuccess ? e : launch_k(kernel, dim3(blocks), dim3(kAttnThreads), smem, s, a);
}

template <typename T, typename CT, int DIM>
cudaError_t launch_plain(const AttnArgs& a, int blocks, cudaStream_t s)
{
    if (a.group <= 2)
        return launch_tiles(k_attn_plain<T, CT, DIM, 2>, a, blocks, PlainShape<T, CT, DIM, 2>::SMEM, s);
    if (a.group <= 8)
        return launch_tiles(k_attn_plain<T, CT, DIM, 8>, a, blocks, PlainShape<T, CT, DIM, 8>::SMEM, s);
    return launch_tiles(k_attn_plain<T, CT, DIM, 16>, a, blocks, PlainShape<T, CT, DIM, 16>::SMEM, s);
}

template <typename T, typename CT>
cudaError_t launch_attention(const AttnArgs& a, int blocks, cudaStream_t s)
{
    const uint64_t joins = static_cast<uint64_t>(a.batch) * a.kv_heads * a.group_blocks * (a.group < kAttnMaxHeads ? a.group : kAttnMaxHeads);
    if (joins > 0x7fffffffull)
        return cudaErrorInvalidConfiguration;
    cudaError_t e = a.head_dim <= 64    ? launch_plain<T, CT, 64>(a, blocks, s)
                    : a.head_dim <= 96  ? launch_plain<T, CT, 96>(a, blocks, s)
                    : a.head_dim <= 128 ? launch_plain<T, CT, 128>(a, blocks, s)
                    : a.head_dim <= 192 ? launch_plain<T, CT, 192>(a, blocks, s)
                                        : launch_plain<T, CT, 256>(a, blocks, s);
    if (e != cudaSuccess)
        return e;
    return launch_k(k_attn_join<T, 32>, dim3(static_cast<unsigned>(joins)), dim3(kAttnThreads), 0, s, a, blocks);
}

}  // namespace ar
