// ar_tree.cuh -- attention of several drafted tokens of each sequence over a
// paged key-value cache: what its kernels have in common.
//
// Work split, as in ar_attn.cuh: an item is one sequence, one key-value head
// and a block of the head's rows (drafted tokens times query heads); its
// cached tokens are cut into tiles, all items' tiles form one line, and each
// block takes an equal run of it.  A block begins at most one item that it
// does not end, and leaves a job for it; items cut by a run's end are joined
// from the blocks' parts, in block order, by k_tree_join.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <climits>

#include "ar_attn.cuh"
#include "ar_kernels.cuh"
#include "ar_launch_k.cuh"
#include "ar_split.h"
#include "ar_tree.h"

namespace ar {

// A sequence: its rows of q, and its cached tokens.
struct TreeSeq {
    int first, n;   // rows first .. first + n - 1 of q
    int context;    // tokens before the drafted ones; below 0 where the length is shorter than they are many
    int end;        // tokens in the cache
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b)
{
    TreeSeq s;
    if (a.seq_start != nullptr) {
        s.first = min(max(a.seq_start[b], 0), a.tokens);
        s.n = max(min(max(a.seq_start[b + 1], 0), a.tokens) - s.first, 0);
    } else {
        s.first = b * a.each;
        s.n = a.each;
    }
    const int length = max(a.lengths[b], 0);
    s.context = length - s.n;
    s.end = min(length, a.capacity);
    return s;
}

// The tokens [start, end) that a block of rows may see, and their tiles: at least one, so that rows without tokens are
// written too.
template <int ROWS, int TILE>
__device__ __forceinline__ Span tree_span(const TreeArgs& a, const TreeSeq& q, int rt)
{
    Span s;
    s.end = q.end;
    int seen = 0;  // drafted tokens that every row of the block sees
    if (a.mask == nullptr) {
        const int last = min((rt + 1) * ROWS, q.n * a.group) - 1;
        seen = rt * ROWS / a.group + 1;
        s.end = max(min(s.end, q.context + last / a.group + 1), 0);
    }
    s.start = a.window > 0 ? static_cast<int>(min(max(static_cast<long long>(q.context) + seen - a.window, 0ll), static_cast<long long>(s.end))) : 0;
    s.tile0 = s.start / TILE;
    s.tiles = max((s.end + TILE - 1) / TILE - s.tile0, 1);
    return s;
}

template <int ROWS>
__device__ __forceinline__ int row_blocks(const TreeArgs& a, const TreeSeq& q) { return (q.n * a.group + ROWS - 1) / ROWS; }

// Tiles of one key-value head of a sequence.
template <int ROWS, int TILE>
__device__ __forceinline__ long long tree_tiles(const TreeArgs& a, const TreeSeq& q)
{
    const int blocks = row_blocks<ROWS>(a, q);
    if (blocks == 0)
        return 0;
    if (a.mask != nullptr)
        return static_cast<long long>(tree_span<ROWS, TILE>(a, q, 0).tiles) * blocks;
    long long sum = 0;
    for (int rt = 0; rt < blocks; ++rt)
        sum += tree_span<ROWS, TILE>(a, q, rt).tiles;
    return sum;
}

// Where a block is on the line.
template <int ROWS, int TILE>
struct TreeCursor {
    int b, h, rt, tile;
    TreeSeq q;
    Span s;
    __device__ __forceinline__ void place(const TreeArgs& a) { s = tree_span<ROWS, TILE>(a, q, rt); }
    // To the next item; there is one.
    __device__ __forceinline__ void next_item(const TreeArgs& a)
    {
        tile = 0;
        if (++rt == row_blocks<ROWS>(a, q)) {
            rt = 0;
            if (++h == a.kv_heads) {
                h = 0;
                do {
                    ++b;
                    q = tree_seq(a, b);
                } while (q.n == 0);
            }
        }
        place(a);
    }
    __device__ __forceinline__ int rows(const TreeArgs& a) const { return min(ROWS, q.n * a.group - rt * ROWS); }
};

// Finds the block's run and its first tile.  All THREADS threads; contains barriers.  s_warp: shared, THREADS / 32 + 2.
template <int ROWS, int TILE, int THREADS>
__device__ Run tree_run(const TreeArgs& a, TreeCursor<ROWS, TILE>& cur, long long* s_warp)
{
    constexpr int WARPS = THREADS / 32;
    long long& s_before = s_warp[WARPS];
    long long& s_b = s_warp[WARPS + 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (a.batch + THREADS - 1) / THREADS, b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    long long mine = 0;
    for (int b = b0; b < b1; ++b)
        mine += tree_tiles<ROWS, TILE>(a, tree_seq(a, b));
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
    for (int w = 0; w < WARPS; ++w) {
        before += w < warp ? s_warp[w] : 0;
        tiles += s_warp[w];
    }
    const Run run = run_of(tiles * a.kv_heads, gridDim.x, blockIdx.x);
    if (run.n == 0)
        return run;
    const long long x = divide(run.lo, a.kv_heads);  // sequence b takes [heads * P, heads * (P + tiles of b)) of the line
    if (before <= x && x < before + mine) {
        int b = b0;
        for (long long n = tree_tiles<ROWS, TILE>(a, tree_seq(a, b)); x >= before + n; n = tree_tiles<ROWS, TILE>(a, tree_seq(a, b))) {
            before += n;
            ++b;
        }
        s_b = b;
        s_before = before;
    }
    __syncthreads();
    cur.b = static_cast<int>(s_b);
    cur.q = tree_seq(a, cur.b);
    const long long each = tree_tiles<ROWS, TILE>(a, cur.q), in = run.lo - s_before * a.kv_heads;
    cur.h = static_cast<int>(divide(in, each));
    long long rest = in - cur.h * each;
    cur.rt = 0;
    cur.place(a);
    if (a.mask != nullptr) {
        cur.rt = static_cast<int>(divide(rest, cur.s.tiles));
        rest -= static_cast<long long>(cur.rt) * cur.s.tiles;
        cur.place(a);
    } else {
        while (rest >= cur.s.tiles) {
            rest -= cur.s.tiles;
            ++cur.rt;
            cur.place(a);
        }
    }
    cur.tile = static_cast<int>(rest);
    return run;
}

// The lower x bits, x of any value.
__device__ __forceinline__ uint32_t low_bits(int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1u; }

// What one row sees: context from first_context on, and the drafted tokens of its mask from first_bit to before last_bit.
struct TreeRow {
    int context, first_context, first_bit, last_bit;
    const uint32_t* mask;  // nullptr: all of them
    int words;

    __device__ __forceinline__ uint32_t word(int w) const { return w >= 0 && w < words ? mask[w] : 0u; }
    // i: the drafted token of the row.
    __device__ void make(const TreeArgs& a, const TreeSeq& q, int i)
    {
        context = q.context;
        first_bit = 0;
        mask = nullptr;
        words = 0;
        int count = i + 1;
        last_bit = i + 1;
        if (a.mask != nullptr) {
            mask = a.mask + static_cast<uint64_t>(q.first + i) * a.mask_words;
            words = a.mask_words;
            last_bit = static_cast<int>(min(static_cast<long long>(q.n), 32ll * words));
            count = 0;
            if (a.window > 0)
                for (int w = 0; w < words; ++w)
                    count += __popc(mask[w] & low_bits(last_bit - 32 * w));
        }
        first_context = 0;
        if (a.window > 0) {
            first_context = static_cast<int>(max(min(static_cast<long long>(context) + count - a.window, static_cast<long long>(context)), 0ll));
            int drop = count - a.window;
            if (drop > 0 && mask == nullptr)
                first_bit = drop;
            if (drop > 0 && mask != nullptr) {
                int w = 0;
                for (int n = __popc(word(w)); drop >= n && w < words; n = __popc(word(w))) {
                    drop -= n;
                    ++w;
                }
                uint32_t left = word(w);
                for (; drop > 0; --drop)
                    left &= left - 1;
                first_bit = 32 * w + __ffs(left) - 1;
            }
        }
    }
    // Which of the 32 tokens from `token` on the row sees.
    __device__ __forceinline__ uint32_t sees(int token) const
    {
        const int o = token - context;  // the first one as a drafted token
        uint32_t bits = low_bits(-o) & ~low_bits(first_context - token);
        if (o > -32) {
            uint32_t drafts = ~0u;
            if (mask != nullptr)
                drafts = __funnelshift_r(word(o >> 5), word((o >> 5) + 1), o & 31);
            bits |= drafts & low_bits(last_bit - o) & ~low_bits(max(first_bit - o, -o));
        }
        return bits;
    }
};

// Whether a tile from `token` on may hold tokens that some row of the sequence sees and another does not.
__device__ __forceinline__ bool tree_mixed(const TreeArgs& a, const TreeSeq& q, int token, int tile)
{
    return token + tile > q.context || (a.window > 0 && token < static_cast<long long>(q.context) + q.n - a.window);
}

// Row r of an item as a row of out and lse.
__device__ __forceinline__ uint64_t tree_out_row(const TreeArgs& a, int first, int head, int row)
{
    const int i = row / a.group, g = row - i * a.group;
    return (static_cast<uint64_t>(first + i) * a.kv_heads + head) * a.group + g;
}

// Writes the job of an item that this block begins and does not end.
template <int ROWS, int TILE>
__device__ __forceinline__ void leave_job(const TreeArgs& a, const TreeCursor<ROWS, TILE>& cur, const Run& run, long long first_tile)
{
    TreeJob job{};
    job.last = block_of(run.total, static_cast<int>(gridDim.x), run.lo + first_tile + cur.s.tiles - 1);
    job.rows = cur.rows(a);
    job.first = cur.q.first;
    job.row0 = cur.rt * ROWS;
    job.head = cur.h;
    a.jobs[blockIdx.x] = job;
}

// ---------------------------------------------------------------------------
// The kernel of multiply-adds, for fp32.  256 threads: half-warp w has rows
// w * RPT .. of ROWS, and its 16 lanes share a tile's 32 tokens, and then the
// head's elements.  A row's maximum, sum and weights stay within its
// half-warp, so the weights meet in shared memory without a block barrier.
// Tiles come by asynchronous copies into a ring, STAGES - 1 of them ahead;
// page numbers a tile earlier still.  Bound by its multiply-adds' loads from
// shared memory: 16 sequences of up to 4096 tokens, 8 heads of 96, 10 rows take
// 148 us for 215 MB (213 us with tiles loaded between the products).
// ---------------------------------------------------------------------------
constexpr int kTreeFmaThreads = 256;

template <int ROWS, int DIM>
struct TreeFmaShape {
    static constexpr int TILE = 32, PITCH = DIM + 4, PPITCH = TILE + 4;
    static constexpr int STAGE = 2 * TILE * PITCH * 4, FIXED = (ROWS * PITCH + ROWS * PPITCH) * 4;
    // Two blocks an SM where three stages of each fit, one otherwise.
    static constexpr int BLOCKS = ROWS == 16 && FIXED + 3 * STAGE <= 112 * 1024 ? 2 : 1;
    static constexpr int FIT = ((BLOCKS == 2 ? 112 : 224) * 1024 - FIXED) / STAGE, STAGES = FIT < 4 ? FIT : 4;
    static_assert(STAGES >= 2, "a tile ahead");
    static constexpr int SMEM = FIXED + STAGES * STAGE;
};

// Four elements of the cache or of q as fp32.
template <typename CT>
__device__ __forceinline__ float4 load_four(const char* p)
{
    if constexpr (sizeof(CT) == 4) {
        return *reinterpret_cast<const float4*>(p);
    } else if constexpr (sizeof(CT) == 2) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        const float2 x = Lanes<CT>::two(w.x), y = Lanes<CT>::two(w.y);
        return make_float4(x.x, x.y, y.x, y.y);
    } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
        const float2 x = Lanes<__half>::two(half2_of_e4m3(w)), y = Lanes<__half>::two(half2_of_e4m3(w >> 16));
        return make_float4(x.x, x.y, y.x, y.y);
    }
}

template <int DIM, int ROWS>
__global__ void __launch_bounds__(kTreeFmaThreads, TreeFmaShape<ROWS, DIM>::BLOCKS)
k_tree_fma(const TreeArgs a)
{
    using P = TreeFmaShape<ROWS, DIM>;
    using Cur = TreeCursor<ROWS, P::TILE>;
    constexpr int TILE = P::TILE, RPT = ROWS / 16, FOURS = DIM / 4, CPT = (FOURS + 15) / 16, STAGES = P::STAGES;
    extern __shared__ __align__(128) char smem[];
    __shared__ uint32_t s_in[STAGES + 1];
    __shared__ int64_t s_offset[STAGES + 1][TILE];
    __shared__ long long s_scan[kTreeFmaThreads / 32 + 2];
    float* const sq = reinterpret_cast<float*>(smem);
    float* const sp = sq + ROWS * P::PITCH;
    char* const stages = smem + P::FIXED;
    pdl_enter();
    const int tid = threadIdx.x, lane = tid & 31, half = tid >> 4, l16 = tid & 15;
    if (tid == 0)
        a.jobs[blockIdx.x].rows = 0;
    Cur cur;
    const Run run = tree_run<ROWS, TILE, kTreeFmaThreads>(a, cur, s_scan);
    const int fours = a.head_dim / 4, n = static_cast<int>(min(run.n, static_cast<long long>(INT_MAX / 2)));
    // The first warp looks pages up, tile `looked` next; all copy, tile `sent` next.
    Cur ahead = cur;
    int looked = 0, sent = 0;
    const auto look = [&] {
        if (looked >= n)
            return;
        if (tid < 32) {
            const int token = (ahead.s.tile0 + ahead.tile) * TILE + lane;
            int page = -1;
            int64_t at = 0;
            if (token >= ahead.s.start && token < ahead.s.end) {
                const uint32_t column = __umulhi(2u * token, a.page_magic) >> a.page_shift;
                page = a.table[static_cast<uint64_t>(ahead.b) * a.table_stride + column];
                if (page >= a.pages)
                    page = -1;
                at = static_cast<int64_t>(static_cast<uint32_t>(page) * a.page_stride +
                                          static_cast<uint32_t>(token - static_cast<int>(column) * a.page_size) * a.token_stride +
                                          static_cast<uint32_t>(ahead.h) * a.head_stride);
            }
            s_offset[looked % (STAGES + 1)][lane] = at;
            const uint32_t in = __ballot_sync(~0u, page >= 0);
            if (lane == 0)
                s_in[looked % (STAGES + 1)] = in;
        }
        if (++looked < n) {
            if (ahead.tile + 1 == ahead.s.tiles)
                ahead.next_item(a);
            else
                ++ahead.tile;
        }
    };
    uint64_t policy;
    asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    const auto send = [&] {  // whose offsets a barrier has shown
        if (sent < n) {
            const uint32_t in = s_in[sent % (STAGES + 1)];
            const uint32_t to = smem_addr(stages + sent % STAGES * P::STAGE);
#pragma unroll 4
            for (int x = tid; x < TILE * FOURS; x += kTreeFmaThreads) {
                const int r = x / FOURS, c = x - r * FOURS;
                const bool read = (in >> r & 1) != 0 && c < fours;
                const int64_t at = read ? s_offset[sent % (STAGES + 1)][r] + 16 * c : 0;
                const uint32_t dst = to + (r * P::PITCH + 4 * c) * 4;
                cp_async16(dst, a.k + at, read, policy);
                cp_async16(dst + TILE * P::PITCH * 4, a.v + at, read, policy);
            }
        }
        ++sent;
        cp_async_commit();
    };
    if (n > 0) {
#pragma unroll 1
        for (int i = 0; i < STAGES; ++i)
            look();
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < STAGES - 1; ++i)
            send();
    }
    float4 o[RPT][CPT];
    float top[RPT], total[RPT];
    TreeRow row[RPT];
    bool valid[RPT], began = false;
    int first = 0;  // the run's tile that the block's part of the item begins with
#pragma unroll 1
    for (int t = 0; t < n; ++t) {
        const int row0 = cur.rt * ROWS, rows = cur.rows(a);
        if (t == 0 || cur.tile == 0) {
            began = cur.tile == 0;
            first = t;
            for (int x = tid; x < ROWS * FOURS; x += kTreeFmaThreads) {
                const int r = x / FOURS, c = x - r * FOURS;
                float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (r < rows && c < fours) {
                    const int i = (row0 + r) / a.group, g = row0 + r - i * a.group;
                    v = *reinterpret_cast<const float4*>(a.q + static_cast<uint64_t>(cur.q.first + i) * a.q_stride +
                                                         (static_cast<uint64_t>(cur.h * a.group + g) * a.head_dim + 4 * c) * sizeof(float));
                }
                *reinterpret_cast<float4*>(sq + r * P::PITCH + 4 * c) = v;
            }
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = half * RPT + i;
                valid[i] = r < rows;
                row[i].make(a, cur.q, (row0 + (valid[i] ? r : 0)) / a.group);
                top[i] = -INFINITY;
                total[i] = 0.0f;
#pragma unroll
                for (int c = 0; c < CPT; ++c)
                    o[i][c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
        }
        cp_async_wait<STAGES - 2>();
        __syncthreads();  // tile t is here, the stage of tile t - 1 and its description are free
        send();
        look();
        const int token0 = (cur.s.tile0 + cur.tile) * TILE;
        const uint32_t in = s_in[t % (STAGES + 1)];
        const float* const sk = reinterpret_cast<const float*>(stages + t % STAGES * P::STAGE);
        const float* const sv = sk + TILE * P::PITCH;
        const bool mixed = tree_mixed(a, cur.q, token0, TILE);
        // Tokens l16 and l16 + 16 of the tile, for the half-warp's rows.
        float2 dot[RPT][2];
#pragma unroll
        for (int i = 0; i < RPT; ++i)
            dot[i][0] = dot[i][1] = make_float2(0.0f, 0.0f);
#pragma unroll 4
        for (int c = 0; c < fours; ++c) {
            const float4 k0 = *reinterpret_cast<const float4*>(sk + l16 * P::PITCH + 4 * c);
            const float4 k1 = *reinterpret_cast<const float4*>(sk + (l16 + 16) * P::PITCH + 4 * c);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const float4 q = *reinterpret_cast<const float4*>(sq + (half * RPT + i) * P::PITCH + 4 * c);
                dot[i][0] = fma2(make_float2(q.x, q.y), make_float2(k0.x, k0.y), dot[i][0]);
                dot[i][0] = fma2(make_float2(q.z, q.w), make_float2(k0.z, k0.w), dot[i][0]);
                dot[i][1] = fma2(make_float2(q.x, q.y), make_float2(k1.x, k1.y), dot[i][1]);
                dot[i][1] = fma2(make_float2(q.z, q.w), make_float2(k1.z, k1.w), dot[i][1]);
            }
        }
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
            const uint32_t sees = mixed ? in & row[i].sees(token0) : in;
            float s[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                s[j] = (dot[i][j].x + dot[i][j].y) * a.scale2;
                if (a.softcap > 0.0f)
                    s[j] = a.softcap2 * tanhf(s[j] * (0.5f * kLn2));
                s[j] = (sees >> (l16 + 16 * j) & 1) != 0 ? s[j] : -INFINITY;
            }
            float best = fmaxf(fmaxf(s[0], s[1]), top[i]);
#pragma unroll
            for (int w = 8; w > 0; w >>= 1)
                best = fmaxf(best, __shfl_xor_sync(~0u, best, w));
            const float base = base_of(best), fix = exp2f(top[i] - base);
            top[i] = best;
            total[i] *= fix;
#pragma unroll
            for (int c = 0; c < CPT; ++c)
                o[i][c] = make_float4(o[i][c].x * fix, o[i][c].y * fix, o[i][c].z * fix, o[i][c].w * fix);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float p = exp2f(s[j] - base);
                total[i] += p;
                // -1: not seen; its value is not even multiplied by 0, whatever it holds
                sp[(half * RPT + i) * P::PPITCH + l16 + 16 * j] = (sees >> (l16 + 16 * j) & 1) != 0 ? p : -1.0f;
            }
        }
        __syncwarp();
        const auto weigh = [&](auto some) {  // some: a weight may be -1
#pragma unroll 4
            for (int j = 0; j < TILE; ++j) {
                float p[RPT];
#pragma unroll
                for (int i = 0; i < RPT; ++i)
                    p[i] = sp[(half * RPT + i) * P::PPITCH + j];
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    const int col = l16 + 16 * c;
                    if (FOURS % 16 == 0 || col < FOURS) {
                        const float4 v = *reinterpret_cast<const float4*>(sv + j * P::PITCH + 4 * col);
#pragma unroll
                        for (int i = 0; i < RPT; ++i)
                            if (!decltype(some)::value || p[i] >= 0.0f) {
                                const float2 x = fma2(make_float2(p[i], p[i]), make_float2(v.x, v.y), make_float2(o[i][c].x, o[i][c].y));
                                const float2 y = fma2(make_float2(p[i], p[i]), make_float2(v.z, v.w), make_float2(o[i][c].z, o[i][c].w));
                                o[i][c] = make_float4(x.x, x.y, y.x, y.y);
                            }
                    }
                }
            }
        };
        if (mixed || in != ~0u)
            weigh(std::true_type{});
        else
            weigh(std::false_type{});
        const bool ends = cur.tile + 1 == cur.s.tiles;
        if (ends || t + 1 == n) {
            const bool whole = began && ends;
            float* const part = a.part + slot_of(static_cast<int>(blockIdx.x), began) * a.slot_floats;
            if (began && !whole && tid == 0)
                leave_job(a, cur, run, first);
#pragma unroll
            for (int i = 0; i < RPT; ++i) {
                const int r = half * RPT + i;
                float sum = total[i];
#pragma unroll
                for (int w = 8; w > 0; w >>= 1)
                    sum += __shfl_xor_sync(~0u, sum, w);
                if (!valid[i])
                    continue;
                const uint64_t out = tree_out_row(a, cur.q.first, cur.h, row0 + r);
#pragma unroll
                for (int c = 0; c < CPT; ++c) {
                    const int col = l16 + 16 * c;
                    if (col >= fours)
                        continue;
                    if (whole)
                        store_four(reinterpret_cast<float*>(a.out) + out * a.head_dim + 4 * col, o[i][c], sum == 0.0f ? 0.0f : a.v_scale / sum);
                    else
                        *reinterpret_cast<float4*>(part + static_cast<uint64_t>(r) * a.head_dim + 4 * col) = o[i][c];
                }
                if (l16 == 0) {
                    if (!whole) {
                        part[static_cast<uint64_t>(a.slot_rows) * a.head_dim + r] = top[i];
                        part[static_cast<uint64_t>(a.slot_rows) * (a.head_dim + 1) + r] = sum;
                    } else if (a.lse != nullptr) {
                        a.lse[out] = lse_of(top[i], sum);
                    }
                }
            }
            __syncthreads();  // the next item's queries come where these are
        }
        if (t + 1 < n) {
            if (ends)
                cur.next_item(a);
            else
                ++cur.tile;
        }
    }
    cp_async_wait<0>();
}

// ---------------------------------------------------------------------------
// The join of the items that several blocks have parts of.  Items of up to
// kFewParts parts take a warp a row, all parts' loads at once; longer ones a
// block a row, whose warps take a part each in turn and meet in shared memory
// in a fixed order.  The rows of all jobs are dealt out evenly to the blocks.
// Bound by its chain of loads, jobs and parts: 5 us (cold) with nothing to
// join, 10 us for 128 items of 64 rows of 128 in two or three parts.  Four blocks an SM: with
// two or eight the whole call is 129 or 126 us in place of 125.
// ---------------------------------------------------------------------------
constexpr int kTreeJoinThreads = 256;
constexpr int kTreeJoinWarps = kTreeJoinThreads / 32;
constexpr int kFewParts = 8;

struct TreeSum {
    float top = -INFINITY, total = 0.0f;
    float4 o[kTreeMaxDim / 128];  // a lane's fours: lane, and lane + 32
    __device__ __forceinline__ TreeSum()
    {
#pragma unroll
        for (int c = 0; c < kTreeMaxDim / 128; ++c)
            o[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    // Adds N parts' values v with references m and sums n.
    template <int N>
    __device__ __forceinline__ void add(const float4 (&v)[N][kTreeMaxDim / 128], const float (&m)[N], const float (&n)[N])
    {
        float best = top;
#pragma unroll
        for (int i = 0; i < N; ++i)
            best = fmaxf(best, m[i]);
        const float base = base_of(best), f = exp2f(top - base);
        top = best;
        total *= f;
#pragma unroll
        for (int c = 0; c < kTreeMaxDim / 128; ++c)
            o[c] = make_float4(o[c].x * f, o[c].y * f, o[c].z * f, o[c].w * f);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float g = exp2f(m[i] - base);
            total = fmaf(n[i], g, total);
#pragma unroll
            for (int c = 0; c < kTreeMaxDim / 128; ++c)
                o[c] = make_float4(fmaf(v[i][c].x, g, o[c].x), fmaf(v[i][c].y, g, o[c].y), fmaf(v[i][c].z, g, o[c].z), fmaf(v[i][c].w, g, o[c].w));
        }
    }
    // Adds parts p, p + step, ... of `parts`, four at once.
    __device__ __forceinline__ void gather(const TreeArgs& a, int first_block, int parts, int row, int p, int step)
    {
        const int lane = threadIdx.x & 31, fours = a.head_dim / 4;
        for (; p < parts; p += 4 * step) {
            float4 v[4][kTreeMaxDim / 128];
            float m[4], n[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int at = p + i * step;
                m[i] = -INFINITY;
                n[i] = 0.0f;
                const float* part = a.part + slot_of(first_block + at, at == 0) * a.slot_floats;  // part 0 begins the item
#pragma unroll
                for (int c = 0; c < kTreeMaxDim / 128; ++c) {
                    v[i][c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    if (at < parts && lane + 32 * c < fours)
                        v[i][c] = *reinterpret_cast<const float4*>(part + static_cast<uint64_t>(row) * a.head_dim + 4 * (lane + 32 * c));
                }
                if (at < parts) {
                    m[i] = part[static_cast<uint64_t>(a.slot_rows) * a.head_dim + row];
                    n[i] = part[static_cast<uint64_t>(a.slot_rows) * (a.head_dim + 1) + row];
                }
            }
            add<4>(v, m, n);
        }
    }
    template <typename T>
    __device__ __forceinline__ void write(const TreeArgs& a, const TreeJob& job, int row) const
    {
        const int lane = threadIdx.x & 31, fours = a.head_dim / 4;
        const uint64_t out = tree_out_row(a, job.first, job.head, job.row0 + row);
#pragma unroll
        for (int c = 0; c < kTreeMaxDim / 128; ++c)
            if (lane + 32 * c < fours)
                store_four(reinterpret_cast<T*>(a.out) + out * a.head_dim + 4 * (lane + 32 * c), o[c], total == 0.0f ? 0.0f : a.v_scale / total);
        if (lane == 0 && a.lse != nullptr)
            a.lse[out] = lse_of(top, total);
    }
};

template <typename T>
__global__ void __launch_bounds__(kTreeJoinThreads)
k_tree_join(const TreeArgs a, const int blocks)
{
    __shared__ int s_few[kTreeMaxBlocks + 1], s_long[kTreeMaxBlocks + 1];  // rows of the jobs before each
    __shared__ TreeJob s_job[kTreeMaxBlocks];
    __shared__ float4 s_o[kTreeJoinWarps][kTreeMaxDim / 4];
    __shared__ float2 s_w[kTreeJoinWarps];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    for (int i = tid; i < blocks; i += kTreeJoinThreads) {
        const TreeJob job = a.jobs[i];
        const bool few = job.last - i < kFewParts;
        s_job[i] = job;
        s_few[i + 1] = few ? job.rows : 0;
        s_long[i + 1] = few ? 0 : job.rows;
    }
    __syncthreads();
    if (warp < 2) {  // running sums, one warp each
        int* const s = warp == 0 ? s_few : s_long;
        int before = 0;
        for (int i0 = 0; i0 < blocks; i0 += 32) {
            int x = i0 + lane < blocks ? s[i0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(~0u, x, o);
                x += lane >= o ? up : 0;
            }
            if (i0 + lane < blocks)
                s[i0 + lane + 1] = before + x;
            before += __shfl_sync(~0u, x, 31);
        }
        if (lane == 0)
            s[0] = 0;
    }
    __syncthreads();
    const auto find = [&](const int* s, int x) {  // the job of row x: the last with s[job] <= x
        int lo = 0, hi = blocks;
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (s[mid] <= x)
                lo = mid;
            else
                hi = mid;
        }
        return lo;
    };
    // Each warp takes rows side by side, most often of one job.
    const int few = s_few[blocks], many = s_long[blocks], warps = gridDim.x * kTreeJoinWarps;
    const int each = (few + warps - 1) / warps, x0 = (blockIdx.x * kTreeJoinWarps + warp) * each, x1 = min(x0 + each, few);
    int j = x0 < x1 ? find(s_few, x0) : 0;
    for (int x = x0; x < x1; ++x) {
        while (s_few[j + 1] <= x)
            ++j;
        TreeSum sum;
        sum.gather(a, j, s_job[j].last - j + 1, x - s_few[j], 0, 1);
        sum.write<T>(a, s_job[j], x - s_few[j]);
    }
    for (int x = blockIdx.x; x < many; x += gridDim.x) {
        const int i = find(s_long, x);
        TreeSum sum;
        sum.gather(a, i, s_job[i].last - i + 1, x - s_long[i], warp, kTreeJoinWarps);
#pragma unroll
        for (int c = 0; c < kTreeMaxDim / 128; ++c)
            s_o[warp][lane + 32 * c] = sum.o[c];
        if (lane == 0)
            s_w[warp] = make_float2(sum.top, sum.total);
        __syncthreads();
        if (warp == 0) {
            for (int w = 1; w < kTreeJoinWarps; w += 1) {
                float4 v[1][kTreeMaxDim / 128];
#pragma unroll
                for (int c = 0; c < kTreeMaxDim / 128; ++c)
                    v[0][c] = s_o[w][lane + 32 * c];
                const float m[1] = {s_w[w].x}, n[1] = {s_w[w].y};
                sum.add<1>(v, m, n);
            }
            sum.write<T>(a, s_job[i], x - s_long[i]);
        }
        __syncthreads();
    }
}

// Launches an attention kernel of `blocks` blocks, with its shared memory limit raised, and the join.
template <typename T, typename... Rest>
cudaError_t launch_tree_kernel(void (*kernel)(TreeArgs, Rest...), const TreeArgs& a, int threads, int smem, int blocks, int sms, cudaStream_t s,
                               const Rest&... rest)
{
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = launch_k(kernel, dim3(blocks), dim3(threads), smem, s, a, rest...);
    if (e != cudaSuccess)
        return e;
    return launch_k(k_tree_join<T>, dim3(sms * 4), dim3(kTreeJoinThreads), 0, s, a, blocks);
}

template <int DIM, int ROWS>
cudaError_t launch_tree_rows(const TreeArgs& a, int most, int sms, cudaStream_t s)
{
    using P = TreeFmaShape<ROWS, DIM>;
    const int blocks = most < P::BLOCKS * sms ? most : P::BLOCKS * sms;
    return launch_tree_kernel<float>(k_tree_fma<DIM, ROWS>, a, kTreeFmaThreads, P::SMEM, blocks, sms, s);
}

template <int DIM>
cudaError_t launch_tree_fma(const TreeArgs& a, const TreeShape& shape, int most, int sms, cudaStream_t s)
{
    return shape.rows == 16 ? launch_tree_rows<DIM, 16>(a, most, sms, s) : launch_tree_rows<DIM, 64>(a, most, sms, s);
}

}  // namespace ar
