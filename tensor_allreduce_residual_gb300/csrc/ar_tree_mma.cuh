// ar_tree_mma.cuh -- attention of drafted tokens over 16-bit and 8-bit caches
// on the fifth-generation tensor core.
//
// A block's tile is 128 rows (drafted tokens times query heads of one
// key-value head; or two such halves) by TOKENS cached tokens.  Scores
// S = Q K^T go from shared memory into tensor memory; a warpgroup for each
// half of the rows, a thread a row, turns them into weights P, which lie in
// tensor memory where the scores lay; O += P V, with O in tensor memory until
// the item's end.  Weights are two 16-bit numbers, their rounding and what it
// leaves, so P V takes two products.
//
//   warps 0 .. 4 NM - 1     softmax, item ends (warp w reads lanes 32 (w % 4) ..)
//   4 warps                 copies: queries, and rings of keys and values
//   1 warp                  allocates tensor memory; one lane issues products
//
// Two score buffers let the next product of scores run while a warpgroup works
// (NM == 1: of alternating tiles, NM == 2: one for each half).  All hand-overs
// are mbarriers.  Waits are bounded: one that gave up is counted, raises the
// block's stop flag, on which all others give up too, and the block leaves.
#pragma once

#include "ar_tcgen05.cuh"
#include "ar_tree.cuh"

namespace ar {

constexpr unsigned long long kTreeWaitLimitNs = 1000000000ull;

// Bounded waits that gave up, in this translation unit's kernels.
static __device__ unsigned int g_tree_wait_timeouts;

__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool bar_test(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}
// Waits until the phase with this parity is complete; false where the block stops.
static __device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, volatile int* stop)
{
    unsigned long long t0, t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
    while (!bar_test(bar, parity)) {
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        if (*stop != 0)
            return false;
        if (t - t0 > kTreeWaitLimitNs) {
            *stop = 1;
            atomicAdd(&g_tree_wait_timeouts, 1u);
            return false;
        }
    }
    return true;
}
__device__ __forceinline__ bool bar_wait_one(uint32_t bar, uint32_t parity, volatile int* stop)
{
    return bar_test(bar, parity) || bar_wait_long(bar, parity, stop);
}
// The same of a whole warp, whose lanes go on, or give up, together.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* stop)
{
    return __all_sync(~0u, bar_wait_one(bar, parity, stop));
}

// The elements of two 16-bit numbers that are infinite or NaN, as a mask of their bits.
template <typename MT>
__device__ __forceinline__ uint32_t not_finite(uint32_t w)
{
    constexpr uint32_t E = std::is_same<MT, __half>::value ? 0x7c00u : 0x7f80u;
    return ((w & E) == E ? 0xffffu : 0u) | ((w & E << 16) == E << 16 ? 0xffff0000u : 0u);
}

enum { kTreeMixed = 16 };  // beside kTileFirst ..

// What the softmax and the products need to know of a tile.
struct TreeTile {
    TreeSeq q;
    int head, row0, rows, token0, flags;
    int b;
    uint32_t valid[4];   // of each copying warp's tokens which are in the cache
    int bad[4];          // whether a value of theirs is infinite or NaN, in a tile that some row sees in part only
};

template <typename T_, typename CT_, int DIM_, int NM_>
struct TreeMmaShape {
    using T = T_;
    using CT = CT_;
    using MT = typename std::conditional<sizeof(CT) == 1, __half, CT>::type;  // of the products' operands
    static constexpr int DIM = DIM_, NM = NM_;
    static constexpr bool SMALL = sizeof(CT) == 1, SCALED = SMALL && !std::is_same<T, __half>::value;
    static constexpr bool BF16 = std::is_same<MT, __nv_bfloat16>::value;
    static constexpr int ROWS = 128 * NM, TOKENS = DIM <= 128 ? 128 : 64, WARP_TOKENS = TOKENS / 4;
    static constexpr int SOFTMAX = 128 * NM, THREADS = SOFTMAX + 128 + 32;
    static constexpr int Q = ROWS * DIM * 2, SLOT = TOKENS * DIM * 2, RAW = SMALL ? TOKENS * DIM : 0;
    // Of a block's 227 KB 1 KB goes to the static arrays, at whose end the dynamic part begins aligned, and 2 KB to barriers.
    static constexpr int MISC = 2048, ROOM = 232448 - 1024 - MISC;
    static constexpr int QS = NM == 1 && DIM <= 128 ? 2 : 1;
    static constexpr int RS = !SMALL ? 0 : DIM == 64 ? 8 : 4;
    static constexpr int FIT = (ROOM - QS * Q - RS * RAW) / SLOT, NS = FIT < 8 ? FIT : 8;
    static_assert(NS >= 3, "a tile's keys and values, and the next one's keys");
    // Fills that are under way before the oldest is waited for.
    static constexpr int LAG = SMALL ? RS - 1 : NS - 2;
    // Descriptions of tiles: of as many as fills may be sent before a tile's last one is handed over, and a tile more.
    static constexpr int TILES = SCALED && DIM > 64 ? 4 : 8;
    static_assert(2 * TILES >= LAG + 3, "a tile is done before its description is wanted again");
    static constexpr int SMEM = QS * Q + NS * SLOT + RS * RAW + MISC;
    // Weights may pass their reference's by 2^AHEAD before it is moved, which costs a pass over O.  fp16 weights are 2^LIFT
    // times as large, so that small ones keep their bits: the largest is 2^15.
    static constexpr float AHEAD = BF16 ? 8.0f : 4.0f, LIFT = BF16 ? 0.0f : 11.0f;
    static constexpr int S_COLUMNS = TOKENS, O_COLUMN = 256;  // score buffers from column 0 on; O of half m at 256 + 128 m
    static_assert(2 * S_COLUMNS <= O_COLUMN && O_COLUMN + NM * (DIM <= 128 ? 128 : 256) <= 512, "tensor memory");
    static constexpr int BARS = 2 * NS + 2 * QS + 2 + 2 + NM + 2 * TILES + 1;
    static_assert(BARS * 8 + 16 + TILES * sizeof(TreeTile) + (SCALED ? QS * ROWS * 4 : 0) <= MISC, "descriptions and barriers");
};

// Shared memory, by address.
template <typename P>
struct TreeSmem {
    char* base;
    uint32_t at;
    __device__ __forceinline__ explicit TreeSmem(char* dynamic)
    {
        at = smem_addr(dynamic);
        base = dynamic;
    }
    static constexpr uint32_t KV = P::QS * P::Q, RAW = KV + P::NS * P::SLOT, BAR = RAW + P::RS * P::RAW, TILE = (BAR + P::BARS * 8 + 15) / 16 * 16,
                              SCALE = TILE + P::TILES * sizeof(TreeTile), END = SCALE + (P::SCALED ? P::QS * P::ROWS * 4 : 0);
    __device__ __forceinline__ uint32_t q(int slot) const { return at + slot * P::Q; }
    __device__ __forceinline__ uint32_t kv(int slot) const { return at + KV + slot * P::SLOT; }
    __device__ __forceinline__ char* raw(int stage) const { return base + RAW + stage * P::RAW; }
    __device__ __forceinline__ uint32_t bar(int i) const { return at + BAR + 8 * i; }
    __device__ __forceinline__ uint32_t kv_full(int s) const { return bar(s); }
    __device__ __forceinline__ uint32_t kv_empty(int s) const { return bar(P::NS + s); }
    __device__ __forceinline__ uint32_t q_full(int s) const { return bar(2 * P::NS + s); }
    __device__ __forceinline__ uint32_t q_empty(int s) const { return bar(2 * P::NS + P::QS + s); }
    __device__ __forceinline__ uint32_t s_full(int s) const { return bar(2 * P::NS + 2 * P::QS + s); }
    __device__ __forceinline__ uint32_t p_ready(int s) const { return bar(2 * P::NS + 2 * P::QS + 2 + s); }
    __device__ __forceinline__ uint32_t o_done(int m) const { return bar(2 * P::NS + 2 * P::QS + 4 + m); }
    __device__ __forceinline__ uint32_t tile_full(int i) const { return bar(2 * P::NS + 2 * P::QS + 4 + P::NM + i); }
    __device__ __forceinline__ uint32_t tile_empty(int i) const { return bar(2 * P::NS + 2 * P::QS + 4 + P::NM + P::TILES + i); }
    __device__ __forceinline__ uint32_t last() const { return bar(P::BARS - 1); }
    __device__ __forceinline__ TreeTile& tile(int t) const { return reinterpret_cast<TreeTile*>(base + TILE)[t % P::TILES]; }
    __device__ __forceinline__ float* scale(int slot) const { return reinterpret_cast<float*>(base + SCALE) + slot * P::ROWS; }
};

// ---------------------------------------------------------------------------
// The copying warps.  Each has a quarter of a tile's tokens.  16-bit elements
// go by asynchronous copies straight to the permuted places that the tensor
// core reads; 8-bit ones to a stage that their own thread then turns into
// fp16, exactly.  Fills (keys, values, keys ..) are handed over in order, LAG
// of them after they were sent on their way.
// ---------------------------------------------------------------------------
template <typename P>
struct TreeFeed {
    using Cur = TreeCursor<P::ROWS, P::TOKENS>;
    static constexpr int CH = P::DIM * static_cast<int>(sizeof(typename P::CT)) / 16, STEPS = P::WARP_TOKENS * CH / 32;
    static_assert(P::WARP_TOKENS * CH % 32 == 0, "whole steps of a warp");
    static constexpr int QCH = P::DIM * 2 / 16;
    const TreeArgs& a;
    const TreeSmem<P>& sm;
    volatile int* stop;
    int warp, lane, chunks, qchunks;
    uint64_t once, often;  // how long L2 keeps lines
    // Where this tile's token of the lane begins in the cache (lanes below WARP_TOKENS), which of them are in it.
    uint32_t off_lo = 0, off_hi = 0, in = 0;
    // The next tile's, while its page number is on its way.
    int page = -1, slot = 0;
    uint32_t head = 0;
    int done = 0;                 // fills handed over
    uint32_t firsts = 0, mixeds = 0;  // bits of the last 32 tiles, by number
    int q_wanted = 0, q_filled = 0, q_handed = 0;  // queries of items: met, sent on their way, handed over

    __device__ TreeFeed(const TreeArgs& a_, const TreeSmem<P>& sm_, volatile int* stop_)
        : a(a_), sm(sm_), stop(stop_), warp((threadIdx.x >> 5) - P::SOFTMAX / 32), lane(threadIdx.x & 31),
          chunks(a_.head_dim * static_cast<int>(sizeof(typename P::CT)) / 16), qchunks(a_.head_dim * 2 / 16)
    {
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(often));
    }
    // A row's 16-byte chunk of an operand of `rows` rows.
    static __device__ __forceinline__ uint32_t place(int row, int c, int rows) { return (c >> 3) * (rows * 128) + row * 128 + ((c ^ row) & 7) * 16; }

    __device__ __forceinline__ void look_up(const Cur& cur)
    {
        const int token = (cur.s.tile0 + cur.tile) * P::TOKENS + warp * P::WARP_TOKENS + lane;
        page = -1;
        if (lane < P::WARP_TOKENS && token >= cur.s.start && token < cur.s.end) {
            const uint32_t column = __umulhi(2u * token, a.page_magic) >> a.page_shift;
            slot = token - static_cast<int>(column) * a.page_size;
            page = a.table[static_cast<uint64_t>(cur.b) * a.table_stride + column];
        }
        head = cur.h;
    }
    __device__ __forceinline__ void found()
    {
        const bool ok = page >= 0 && page < a.pages;
        const uint64_t off = ok ? static_cast<uint32_t>(page) * a.page_stride + static_cast<uint32_t>(slot) * a.token_stride + head * a.head_stride : 0;
        off_lo = static_cast<uint32_t>(off);
        off_hi = static_cast<uint32_t>(off >> 32);
        in = __ballot_sync(~0u, ok);
    }
    // The queries of an item, as its rows, to their slot, which is free.  LATE: they are there on return.
    template <bool LATE>
    __device__ __forceinline__ void queries(const TreeSeq& q, int h, int row0, int rows)
    {
        const int s = q_filled++ % P::QS;
        const uint32_t to = sm.q(s);
        if constexpr (!P::SCALED) {
#pragma unroll 8
            for (int x = warp * 32 + lane; x < P::ROWS * QCH; x += 128) {
                const int row = x / QCH, c = x - row * QCH, i = (row0 + row) / a.group, g = row0 + row - i * a.group;
                const bool read = row < rows && c < qchunks;
                const char* from = a.q;
                if (read)
                    from += static_cast<uint64_t>(q.first + i) * a.q_stride + (static_cast<uint64_t>(h) * a.group + g) * a.head_dim * 2 + c * 16;
                const uint32_t dst = (row >> 7) * (128 * P::DIM * 2) + place(row & 127, c, 128);
                if constexpr (LATE)
                    *reinterpret_cast<uint4*>(sm.base + (to - sm.at) + dst) = read ? *reinterpret_cast<const uint4*>(from) : make_uint4(0, 0, 0, 0);
                else
                    cp_async16(to + dst, from, read);
            }
        } else {
            // bf16 queries on an 8-bit cache: scaled by a power of two a row, so that the largest element becomes 2^14 or more
            // and those down to 2^-28 of it keep all their bits in fp16.
            float* const scale = sm.scale(s);
#pragma unroll 4
            for (int row = warp; row < P::ROWS; row += 4) {
                const int i = (row0 + row) / a.group, g = row0 + row - i * a.group;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (row < rows && lane < qchunks)
                    w = *reinterpret_cast<const uint4*>(a.q + static_cast<uint64_t>(q.first + i) * a.q_stride +
                                                        (static_cast<uint64_t>(h) * a.group + g) * a.head_dim * 2 + lane * 16);
                const float2 f[4] = {Lanes<typename P::T>::two(w.x), Lanes<typename P::T>::two(w.y), Lanes<typename P::T>::two(w.z),
                                     Lanes<typename P::T>::two(w.w)};
                float most = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    most = fmaxf(most, fmaxf(fabsf(f[k].x), fabsf(f[k].y)));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1)
                    most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
                const int e = max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -112) - 14;
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                if (lane < QCH) {
                    uint4 x;
                    x.x = Lanes<__half>::word(f[0].x * down, f[0].y * down);
                    x.y = Lanes<__half>::word(f[1].x * down, f[1].y * down);
                    x.z = Lanes<__half>::word(f[2].x * down, f[2].y * down);
                    x.w = Lanes<__half>::word(f[3].x * down, f[3].y * down);
                    *reinterpret_cast<uint4*>(sm.base + (to - sm.at) + (row >> 7) * (128 * P::DIM * 2) + place(row & 127, lane, 128)) = x;
                }
                if (lane == 0)  // finite: an infinite factor would make the scores of keys that are 0 NaN
                    scale[row] = fmaxf(fminf(ldexpf(a.scale2, e), FLT_MAX), -FLT_MAX);
            }
        }
    }
    __device__ __forceinline__ uint32_t q_phase() const { return (q_filled / P::QS & 1) ^ 1; }
    // Sends fill f (of keys or of values) on its way.
    __device__ __forceinline__ bool send(int f, const char* from, uint64_t policy)
    {
        uint32_t to;
        if constexpr (P::SMALL) {
            to = smem_addr(sm.raw(f % P::RS));
        } else {
            if (!bar_wait(sm.kv_empty(f % P::NS), (f / P::NS & 1) ^ 1, stop))
                return false;
            to = sm.kv(f % P::NS);
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int row = (lane + 32 * i) / CH, c = lane + 32 * i - row * CH;
            const uint32_t lo = __shfl_sync(~0u, off_lo, row), hi = __shfl_sync(~0u, off_hi, row);
            const bool read = (in >> row & 1) != 0 && c < chunks;
            const uint64_t at = read ? (static_cast<uint64_t>(hi) << 32 | lo) + c * 16 : 0;
            // an 8-bit chunk lies where its own thread finds it
            const uint32_t dst = P::SMALL ? to + (i * 128 + warp * 32 + lane) * 16 : to + place(warp * P::WARP_TOKENS + row, c, P::TOKENS);
            cp_async16(dst, from + at, read, policy);
        }
        cp_async_commit();
        return true;
    }
    // Hands over the oldest fill, whose copies have arrived.
    __device__ __forceinline__ bool hand_over()
    {
        const int f = done++, t = f >> 1;
        const bool values = f & 1, mixed = values && (mixeds >> (t & 31) & 1) != 0, first = !values && (firsts >> (t & 31) & 1) != 0;
        if (first && q_filled == q_handed) {
            // The queries' slot was not free when the keys were sent.  It is when what was handed over before has been used.
            if (!bar_wait(sm.q_empty(q_filled % P::QS), q_phase(), stop) || !bar_wait(sm.tile_full(t % P::TILES), t / P::TILES & 1, stop))
                return false;
            const TreeTile& tile = sm.tile(t);
            queries<true>(tile.q, tile.head, tile.row0, tile.rows);
        }
        char* const to = sm.base + (sm.kv(f % P::NS) - sm.at);
        bool bad = false;
        if constexpr (P::SMALL) {
            if (!bar_wait(sm.kv_empty(f % P::NS), (f / P::NS & 1) ^ 1, stop))
                return false;
            const char* const raw = sm.raw(f % P::RS);
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int row = (lane + 32 * i) / CH, c = lane + 32 * i - row * CH;
                const uint4 w = *reinterpret_cast<const uint4*>(raw + (i * 128 + warp * 32 + lane) * 16);
                uint32_t h[8] = {half2_of_e4m3(w.x), half2_of_e4m3(w.x >> 16), half2_of_e4m3(w.y), half2_of_e4m3(w.y >> 16),
                                 half2_of_e4m3(w.z), half2_of_e4m3(w.z >> 16), half2_of_e4m3(w.w), half2_of_e4m3(w.w >> 16)};
                if (mixed) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t x = not_finite<__half>(h[k]);
                        bad = bad || x != 0;
                        h[k] &= ~x;
                    }
                }
                const int r = warp * P::WARP_TOKENS + row;
                *reinterpret_cast<uint4*>(to + place(r, 2 * c, P::TOKENS)) = make_uint4(h[0], h[1], h[2], h[3]);
                *reinterpret_cast<uint4*>(to + place(r, 2 * c + 1, P::TOKENS)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
        } else if (mixed) {
#pragma unroll 4
            for (int i = 0; i < STEPS; ++i) {
                const int row = (lane + 32 * i) / CH, c = lane + 32 * i - row * CH;
                uint4* const p = reinterpret_cast<uint4*>(to + place(warp * P::WARP_TOKENS + row, c, P::TOKENS));
                const uint4 w = *p;
                const uint4 x = make_uint4(not_finite<typename P::MT>(w.x), not_finite<typename P::MT>(w.y), not_finite<typename P::MT>(w.z),
                                           not_finite<typename P::MT>(w.w));
                if ((x.x | x.y | x.z | x.w) != 0) {
                    bad = true;
                    *p = make_uint4(w.x & ~x.x, w.y & ~x.y, w.z & ~x.z, w.w & ~x.w);
                }
            }
        }
        if (bad)
            sm.tile(t).bad[warp] = 1;
        fence_async_proxy();
        __syncwarp();
        if (lane == 0) {
            if (first)
                bar_arrive(sm.q_full(q_handed % P::QS));
            bar_arrive(sm.kv_full(f % P::NS));
        }
        q_handed += first;
        return true;
    }
    __device__ bool run(Cur cur, const Run& line, int n)
    {
        look_up(cur);
        bool first = true;
        for (int t = 0; t < n; ++t) {
            found();
            const bool begins = cur.tile == 0, ends = cur.tile + 1 == cur.s.tiles;
            const int token0 = (cur.s.tile0 + cur.tile) * P::TOKENS;
            const bool mixed = tree_mixed(a, cur.q, token0, P::TOKENS);
            first = first || begins;
            if (!bar_wait(sm.tile_empty(t % P::TILES), (t / P::TILES & 1) ^ 1, stop))
                return false;
            TreeTile& tile = sm.tile(t);
            if (lane == 0) {
                tile.valid[warp] = in;
                tile.bad[warp] = 0;
                if (warp == 0) {
                    tile.q = cur.q;
                    tile.head = cur.h;
                    tile.row0 = cur.rt * P::ROWS;
                    tile.rows = cur.rows(a);
                    tile.token0 = token0;
                    tile.b = cur.b;
                    tile.flags = (first ? kTileFirst : 0) | (ends || t + 1 == n ? kTileLast : 0) | (begins ? kTileBegins : 0) | (ends ? kTileEnds : 0) |
                                 (mixed ? kTreeMixed : 0);
                    if (begins && n - t < cur.s.tiles)
                        leave_job(a, cur, line, t);
                }
                bar_arrive(sm.tile_full(t % P::TILES));
            }
            firsts = (firsts & ~(1u << (t & 31))) | (first ? 1u : 0u) << (t & 31);
            mixeds = (mixeds & ~(1u << (t & 31))) | (mixed ? 1u : 0u) << (t & 31);
            // The queries go with the keys where their slot is free and those of no earlier item wait for one.
            if (first) {
                ++q_wanted;
                if (q_filled + 1 == q_wanted && __all_sync(~0u, bar_test(sm.q_empty(q_filled % P::QS), q_phase())))
                    queries<false>(cur.q, cur.h, cur.rt * P::ROWS, cur.rows(a));
            }
            const uint64_t policy = row_blocks<P::ROWS>(a, cur.q) == 1 ? once : often;
            first = false;
            if (t + 1 < n) {
                if (ends)
                    cur.next_item(a);
                else
                    ++cur.tile;
                look_up(cur);
            }
            for (int f = 2 * t; f < 2 * t + 2; ++f) {
                if (!send(f, f & 1 ? a.v : a.k, policy))
                    return false;
                if (f - done >= P::LAG) {
                    cp_async_wait<P::LAG>();
                    if (!hand_over())
                        return false;
                }
            }
        }
        cp_async_wait<0>();
        while (done < 2 * n)
            if (!hand_over())
                return false;
        return true;
    }
};

// ---------------------------------------------------------------------------
// The products, issued by one thread: scores of step u + 1, then the weighted
// values of step u, a step being a half of the rows of a tile.
// ---------------------------------------------------------------------------
template <typename P>
__device__ bool tree_products(const TreeArgs& a, const TreeSmem<P>& sm, uint32_t tmem, int n, volatile int* stop)
{
    const int ksteps = (a.head_dim + 15) / 16;
    const uint32_t desc_s = product_desc(P::BF16, P::TOKENS, false), desc_o = product_desc(P::BF16, 16 * ksteps, true);
    const int steps = n * P::NM;
    int items = 0;        // whose queries have been waited for
    uint32_t firsts = 0;  // which of the last tiles begin the block's part of an item, by number
    const auto scores = [&](int u) {
        const int t = u / P::NM, m = u % P::NM, s = 2 * t % P::NS;
        if (m == 0) {
            if (!bar_wait_one(sm.tile_full(t % P::TILES), t / P::TILES & 1, stop))
                return false;
            const bool first = sm.tile(t).flags & kTileFirst;
            firsts = (firsts & ~(1u << (t & 31))) | (first ? 1u : 0u) << (t & 31);
            if (first) {
                if (!bar_wait_one(sm.q_full(items % P::QS), items / P::QS & 1, stop))
                    return false;
                ++items;
            }
            if (!bar_wait_one(sm.kv_full(s), 2 * t / P::NS & 1, stop))
                return false;
        }
        const int flags = sm.tile(t).flags;
        tcgen05_after_sync();
        const uint32_t q = sm.q((items - 1) % P::QS) + m * (128 * P::DIM * 2), k = sm.kv(s), d = tmem + (u & 1) * P::S_COLUMNS;
        for (int j = 0; j < ksteps; ++j)
            mma_shared(d, operand_desc(q + (j >> 2) * (128 * 128) + (j & 3) * 32, 16, 1024), operand_desc(k + (j >> 2) * (P::TOKENS * 128) + (j & 3) * 32, 16, 1024),
                       desc_s, j > 0);
        tcgen05_commit(sm.s_full(u & 1));
        if (m == P::NM - 1) {
            tcgen05_commit(sm.kv_empty(s));
            if (flags & kTileLast)
                tcgen05_commit(sm.q_empty((items - 1) % P::QS));
        }
        return true;
    };
    if (!scores(0))
        return false;
    for (int u = 0; u < steps; ++u) {
        const int t = u / P::NM, m = u % P::NM, f = 2 * t + 1, s = f % P::NS;
        const bool begins = firsts >> (t & 31) & 1;
        if (u + 1 < steps) {
            // The scores' buffer holds the weights of step u - 1 until its product is done.
            if (u > 0 && !bar_wait_one(sm.o_done((u - 1) % P::NM), (u - 1) / P::NM & 1, stop))
                return false;
            if (!scores(u + 1))
                return false;
        }
        if (!bar_wait_one(sm.p_ready(u & 1), u >> 1 & 1, stop))
            return false;
        if (m == 0 && !bar_wait_one(sm.kv_full(s), f / P::NS & 1, stop))
            return false;
        tcgen05_after_sync();
        const uint32_t p = tmem + (u & 1) * P::S_COLUMNS, o = tmem + P::O_COLUMN + m * 128, v = sm.kv(s);
        for (int j = 0; j < P::TOKENS / 16; ++j) {
            const uint64_t b = operand_desc(v + j * 2048, P::TOKENS * 128, 1024);
            const uint32_t w = p + (j >> 1) * 32 + (j & 1) * 8;  // of 32 tokens 16 columns of weights, then 16 of what they leave
            mma_tensor(o, w, b, desc_o, !(begins && j == 0));
            mma_tensor(o, w + 16, b, desc_o, true);
        }
        tcgen05_commit(sm.o_done(m));
        if (m == P::NM - 1)
            tcgen05_commit(sm.kv_empty(s));
    }
    return true;
}

// ---------------------------------------------------------------------------
// The softmax: a thread has a row.
// ---------------------------------------------------------------------------
template <typename P>
struct TreeSoft {
    using T = typename P::T;
    using MT = typename P::MT;
    const TreeArgs& a;
    const TreeSmem<P>& sm;
    volatile int* stop;
    int m, row, lane;
    uint32_t lanes;  // the warp's lanes in an address of tensor memory
    uint32_t o;
    float factor = 0.0f, reference = -INFINITY, total = 0.0f;
    TreeRow sees;

    __device__ TreeSoft(const TreeArgs& a_, const TreeSmem<P>& sm_, uint32_t tmem, volatile int* stop_) : a(a_), sm(sm_), stop(stop_)
    {
        const int warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        m = warp >> 2;
        row = threadIdx.x;  // of the item
        lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        o = tmem + lanes + P::O_COLUMN + m * 128;
    }
    static __device__ __forceinline__ uint32_t valid_word(const TreeTile& tile, int c)
    {
        if constexpr (P::WARP_TOKENS == 32)
            return tile.valid[c];
        else
            return tile.valid[2 * c] | tile.valid[2 * c + 1] << 16;
    }
    // Which of 32 tokens of a tile the row sees.
    __device__ __forceinline__ uint32_t seen(const TreeTile& tile, int c) const
    {
        const uint32_t word = valid_word(tile, c);
        return tile.flags & kTreeMixed ? word & sees.sees(tile.token0 + 32 * c) : word;
    }
    // Weights of a tile whose scores lie at `s`.  PART: not every row sees every token.  CAP: with softcap.  One loop over
    // groups of 32 tokens, not unrolled: the four warps' instructions have to stay in the cache.
    template <bool PART, bool CAP>
    __device__ __forceinline__ bool weights(const TreeTile& tile, uint32_t s, bool first, int t)
    {
        constexpr int CHUNKS = P::TOKENS / 32;
        float most = -INFINITY;
#pragma unroll 1
        for (int c = 0; c < CHUNKS; ++c) {
            const uint32_t word = PART ? seen(tile, c) : ~0u;
            uint32_t x[32];
            tmem_load32(s + 32 * c, x);
            tcgen05_wait_load();
            float part[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float y = __uint_as_float(x[i]) * factor;
                part[i & 3] = fmaxf(part[i & 3], !PART || (word >> i & 1) != 0 ? y : -INFINITY);
            }
            most = fmaxf(most, fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])));
        }
        if (CAP && most != -INFINITY)
            most = a.softcap2 * tanh_fast(most);  // which rises with its argument
        // The reference is moved where weights would pass it by 2^AHEAD, and with it what is summed up so far.
        const float before = reference;
        if (first || most - P::LIFT > reference + P::AHEAD)
            reference = most - P::LIFT;
        if (!first && __any_sync(~0u, reference != before)) {
            if (!bar_wait(sm.o_done(m), (t - 1) & 1, stop))
                return false;
            tcgen05_after_sync();
            const float fix = reference == before ? 1.0f : exp2_fast(before - reference);
            total *= fix;
#pragma unroll 1
            for (int c = 0; c < a.head_dim; c += 32) {
                uint32_t x[32];
                tmem_load32(o + c, x);
                tcgen05_wait_load();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    x[i] = __float_as_uint(__uint_as_float(x[i]) * fix);
                tmem_store32(o + c, x);
            }
        }
        const float base = base_of(reference);
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 1
        for (int c = 0; c < CHUNKS; ++c) {
            const uint32_t word = PART ? seen(tile, c) : ~0u;
            uint32_t x[32], w[32];
            tmem_load32(s + 32 * c, x);
            tcgen05_wait_load();
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
                float p[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float z = __uint_as_float(x[i + j]);
                    const float y = CAP ? a.softcap2 * tanh_fast(z * factor) - base : fmaf(z, factor, -base);
                    p[j] = exp2_fast(!PART || (word >> (i + j) & 1) != 0 ? y : -INFINITY);
                    sum[i & 2 ? 2 + j : j] += p[j];
                }
                const uint32_t high = Lanes<MT>::word(p[0], p[1]);
                const float2 back = Lanes<MT>::two(high);
                w[i / 2] = high;
                w[16 + i / 2] = Lanes<MT>::word(p[0] - back.x, p[1] - back.y);
            }
            tmem_store32(s + 32 * c, w);
        }
        total += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        tcgen05_wait_store();
        return true;
    }
    __device__ __forceinline__ bool weights(const TreeTile& tile, uint32_t s, bool first, int t, bool part)
    {
        if (a.softcap > 0.0f)
            return weights<true, true>(tile, s, first, t);
        return part ? weights<true, false>(tile, s, first, t) : weights<false, false>(tile, s, first, t);
    }
    // Waits for tile t's product with the values; the one before was waited for already.
    __device__ __forceinline__ bool weighted(int t)
    {
        if (!bar_wait(sm.o_done(m), t & 1, stop))
            return false;
        tcgen05_after_sync();
        return true;
    }
    // Values that are infinite or NaN, in a tile that rows see in part: the product took 0 for them, and the rows that see
    // them get them here, out of the cache once more.
    __device__ __forceinline__ bool poison(const TreeTile& tile, int t, bool valid)
    {
        if (!weighted(t))
            return false;
#pragma unroll 1
        for (int c0 = 0; c0 < a.head_dim; c0 += 32) {
            float add[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
                add[i] = 0.0f;
#pragma unroll 1
            for (int c = 0; c < P::TOKENS / 32 && valid; ++c) {
#pragma unroll 1
                for (uint32_t word = valid_word(tile, c) & sees.sees(tile.token0 + 32 * c); word != 0; word &= word - 1) {
                    const int token = tile.token0 + 32 * c + __ffs(word) - 1;
                    const uint32_t column = __umulhi(2u * token, a.page_magic) >> a.page_shift;
                    const int page = a.table[static_cast<uint64_t>(tile.b) * a.table_stride + column];
                    const char* const v = a.v + static_cast<uint32_t>(page) * a.page_stride +
                                          static_cast<uint32_t>(token - static_cast<int>(column) * a.page_size) * a.token_stride +
                                          static_cast<uint32_t>(tile.head) * a.head_stride;
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (c0 + i < a.head_dim) {
                            const float4 x = load_four<typename P::CT>(v + (c0 + i) * sizeof(typename P::CT));
                            add[i] += isfinite(x.x) ? 0.0f : x.x;
                            add[i + 1] += isfinite(x.y) ? 0.0f : x.y;
                            add[i + 2] += isfinite(x.z) ? 0.0f : x.z;
                            add[i + 3] += isfinite(x.w) ? 0.0f : x.w;
                        }
                }
            }
            __syncwarp();
            uint32_t x[32];
            tmem_load32(o + c0, x);
            tcgen05_wait_load();
#pragma unroll
            for (int i = 0; i < 32; ++i)
                x[i] = __float_as_uint(__uint_as_float(x[i]) + add[i]);
            tmem_store32(o + c0, x);
        }
        tcgen05_wait_store();
        tcgen05_before_sync();
        return true;
    }
    // The end of the block's part of an item: the result, or the part.
    __device__ __forceinline__ bool finish(const TreeTile& tile, int t, bool began, bool any, bool valid)
    {
        if (!weighted(t))
            return false;
        if (!any)
            return true;
        const bool whole = began && (tile.flags & kTileEnds);
        const uint64_t out = valid ? tree_out_row(a, tile.q.first, tile.head, tile.row0 + row) : 0;
        float* const part = a.part + slot_of(static_cast<int>(blockIdx.x), began) * a.slot_floats;
        const float f = total == 0.0f ? 0.0f : a.v_scale / total;
#pragma unroll 1
        for (int c = 0; c < a.head_dim; c += 32) {
            uint32_t x[32];
            tmem_load32(o + c, x);
            tcgen05_wait_load();
            if (!valid)
                continue;
            if (whole) {
                T* const to = reinterpret_cast<T*>(a.out) + out * a.head_dim + c;
#pragma unroll
                for (int i = 0; i < 32; i += 8)
                    if (c + i < a.head_dim) {
                        uint4 w;
                        w.x = Lanes<T>::word(__uint_as_float(x[i]) * f, __uint_as_float(x[i + 1]) * f);
                        w.y = Lanes<T>::word(__uint_as_float(x[i + 2]) * f, __uint_as_float(x[i + 3]) * f);
                        w.z = Lanes<T>::word(__uint_as_float(x[i + 4]) * f, __uint_as_float(x[i + 5]) * f);
                        w.w = Lanes<T>::word(__uint_as_float(x[i + 6]) * f, __uint_as_float(x[i + 7]) * f);
                        *reinterpret_cast<uint4*>(to + i) = w;
                    }
            } else {
                float* const to = part + static_cast<uint64_t>(row) * a.head_dim + c;
#pragma unroll
                for (int i = 0; i < 32; i += 4)
                    if (c + i < a.head_dim)
                        *reinterpret_cast<uint4*>(to + i) = make_uint4(x[i], x[i + 1], x[i + 2], x[i + 3]);
            }
        }
        if (valid && whole && a.lse != nullptr)
            a.lse[out] = lse_of(reference, total);
        if (valid && !whole) {
            part[static_cast<uint64_t>(a.slot_rows) * a.head_dim + row] = reference;
            part[static_cast<uint64_t>(a.slot_rows) * (a.head_dim + 1) + row] = total;
        }
        return true;
    }
    __device__ bool run(uint32_t tmem, int n)
    {
        bool began = false, valid = false, any = false;
        int items = 0;
        for (int t = 0; t < n; ++t) {
            if (!bar_wait(sm.tile_full(t % P::TILES), t / P::TILES & 1, stop))
                return false;
            const TreeTile& tile = sm.tile(t);
            const int flags = tile.flags;
            const bool first = flags & kTileFirst;
            const int u = t * P::NM + m;
            if (!bar_wait(sm.s_full(u & 1), u >> 1 & 1, stop))
                return false;
            tcgen05_after_sync();
            if (first) {
                began = flags & kTileBegins;
                valid = row < tile.rows;
                any = __any_sync(~0u, valid);
                sees.make(a, tile.q, (tile.row0 + (valid ? row : 0)) / a.group);
                reference = -INFINITY;
                total = 0.0f;
                factor = a.scale2;
                if constexpr (P::SCALED) {
                    if (!bar_wait(sm.q_full(items % P::QS), items / P::QS & 1, stop))
                        return false;
                    factor = sm.scale(items % P::QS)[row];
                    __syncwarp();
                    if (lane == 0)
                        bar_arrive(sm.q_empty(items % P::QS));
                }
                ++items;
            }
            if (any) {
                bool part = flags & kTreeMixed;
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    part = part || tile.valid[w] != (P::WARP_TOKENS == 32 ? ~0u : 0xffffu);
                const uint32_t s = tmem + lanes + (u & 1) * P::S_COLUMNS;
                if (!weights(tile, s, first, t, part))
                    return false;
            }
            bool bad = false;
            if (flags & kTreeMixed) {  // the values have to be there first; once the weights are, their slot may be filled anew
                const int f = 2 * t + 1;
                if (!bar_wait(sm.kv_full(f % P::NS), f / P::NS & 1, stop))
                    return false;
                const volatile int* const found = tile.bad;
                bad = any && (found[0] | found[1] | found[2] | found[3]) != 0;
            }
            // A parity tells two phases apart only: the last product has to be seen done before the next can be.
            if (t > 0 && !bar_wait(sm.o_done(m), (t - 1) & 1, stop))
                return false;
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0)
                bar_arrive(sm.p_ready(u & 1));
            if (bad && !poison(tile, t, valid))
                return false;
            if ((flags & kTileLast) && !finish(tile, t, began, any, valid))
                return false;
            __syncwarp();
            if (lane == 0)
                bar_arrive(sm.tile_empty(t % P::TILES));
        }
        return true;
    }
};

template <typename P>
__global__ void __launch_bounds__(P::THREADS, 1)
k_tree_mma(const TreeArgs a)
{
    extern __shared__ __align__(1024) char dynamic[];
    __shared__ uint32_t s_tmem;
    __shared__ int s_stop;
    static_assert(TreeSmem<P>::END <= P::SMEM, "shared memory");
    pdl_enter();
    const TreeSmem<P> sm(dynamic);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int COPY = P::SOFTMAX / 32, ISSUE = COPY + 4;
    if (warp == ISSUE)
        tmem_alloc(smem_addr(&s_tmem), 512);
    if (threadIdx.x == 0) {
        s_stop = 0;
        for (int i = 0; i < P::NS; ++i) {
            bar_init(sm.kv_full(i), 4);
            bar_init(sm.kv_empty(i), 1);
        }
        for (int i = 0; i < P::QS; ++i) {
            bar_init(sm.q_full(i), 4);
            bar_init(sm.q_empty(i), P::SCALED ? 1 + P::SOFTMAX / 32 : 1);  // the product's, and the factors' readers
        }
        for (int i = 0; i < 2; ++i) {
            bar_init(sm.s_full(i), 1);
            bar_init(sm.p_ready(i), 4);
        }
        for (int i = 0; i < P::NM; ++i)
            bar_init(sm.o_done(i), 1);
        for (int i = 0; i < P::TILES; ++i) {
            bar_init(sm.tile_full(i), 4);
            bar_init(sm.tile_empty(i), P::SOFTMAX / 32);
        }
        bar_init(sm.last(), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        a.jobs[blockIdx.x].rows = 0;
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = s_tmem;
    volatile int* const stop = &s_stop;
    TreeCursor<P::ROWS, P::TOKENS> cur;
    const Run line = tree_run<P::ROWS, P::TOKENS, P::THREADS>(a, cur);  // the job's 0 is written before: it contains a barrier
    const int n = static_cast<int>(min(line.n, static_cast<long long>(INT_MAX / 4)));
    if (n > 0) {
        if (warp == ISSUE) {
            if (lane == 0 && !tree_products<P>(a, sm, tmem, n, stop)) {
                // Stopped: the products under way end before shared and tensor memory are given back.
                tcgen05_commit(sm.last());
                unsigned long long t0, t;
                asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
                do
                    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
                while (!bar_test(sm.last(), 0) && t - t0 < kTreeWaitLimitNs);
            }
            __syncwarp();
        } else if (warp >= COPY) {
            TreeFeed<P> feed(a, sm, stop);
            if (!feed.run(cur, line, n))
                cp_async_wait<0>();
            __syncwarp();
        } else {
            TreeSoft<P> soft(a, sm, tmem, stop);
            soft.run(tmem, n);
            __syncwarp();
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    if (warp == ISSUE)
        tmem_free(tmem, 512);
}

// What this translation unit's kernels gave up waiting for since the last time.
template <typename T>
cudaError_t take_tree_wait_timeouts(unsigned int* count)
{
    unsigned int v = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_tree_wait_timeouts, sizeof(v));
    if (e == cudaSuccess && v != 0) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_tree_wait_timeouts, &zero, sizeof(zero));
    }
    *count = v;
    return e;
}

template <typename T, typename CT, int DIM>
cudaError_t launch_tree_mma(const TreeArgs& a, const TreeShape& shape, int most, int sms, cudaStream_t s)
{
    const int blocks = most < sms ? most : sms;
    if constexpr (DIM <= 128) {
        if (shape.rows == 256) {
            using P = TreeMmaShape<T, CT, DIM, 2>;
            return launch_tree_kernel<T>(k_tree_mma<P>, a, P::THREADS, P::SMEM, blocks, sms, s);
        }
    }
    using P = TreeMmaShape<T, CT, DIM, 1>;
    return launch_tree_kernel<T>(k_tree_mma<P>, a, P::THREADS, P::SMEM, blocks, sms, s);
}

template <typename T, typename CT>
cudaError_t launch_tree(const TreeArgs& a, const TreeShape& shape, int most, int sms, cudaStream_t s)
{
    return a.head_dim <= 64    ? launch_tree_mma<T, CT, 64>(a, shape, most, sms, s)
           : a.head_dim <= 128 ? launch_tree_mma<T, CT, 128>(a, shape, most, sms, s)
           : a.head_dim <= 192 ? launch_tree_mma<T, CT, 192>(a, shape, most, sms, s)
                               : launch_tree_mma<T, CT, 256>(a, shape, most, sms, s);
}

}  // namespace ar
