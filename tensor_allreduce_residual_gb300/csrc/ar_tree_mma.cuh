// ar_tree_mma.cuh -- attention of drafted tokens over 16-bit and 8-bit caches
// on the fifth-generation tensor core.
//
// A block's tile is 128 rows (drafted tokens times query heads of one
// key-value head; or two such halves) by TOKENS cached tokens.  Scores
// S = Q K^T go from shared memory into tensor memory; a thread a row turns
// them into weights P, which lie in tensor memory where the scores lay;
// O += P V, with O in tensor memory until the item's end.  Weights are two
// 16-bit numbers, their rounding and what it leaves, so P V takes two products.
//
//   8 softmax warps (4 for heads over 128), a thread a row
//   4 helping warps: queries, what tensor copies cannot bring, 8-bit to fp16;
//     where pages do not fit boxes, keys and values as well (TreeFeed)
//   2 warps that issue products: scores, weighted values
//   2 warps that ask for tensor copies: keys, values (TreeBoxes)
//
// A softmax step takes a warpgroup longer than a tile of bf16 takes from HBM,
// so heads of up to 128 have two warpgroups, with a score buffer and an O
// each: with 256 rows (NM == 2) they have a half of the rows each, with up to
// 128 (NM == 1) alternate tiles, whose two O's are joined at the item's end.
// Blocks take equal runs of tiles over all items; an item that several blocks
// have is joined by k_tree_join.
//
// What bounds it: 64 sequences of 8192 cached tokens (537 MB of bf16, 64 rows)
// take 125 us with the join.  A block takes a tile in 1.45 us there, which is
// 6.8 TB/s, HBM's rate, for 78 us; the rest is the start (3 us, the first
// tile's way through tensor memory 4 to 9 us), the last tile's softmax and
// O (5 us), and the join (10 us).  With 256 rows a group's way round, scores,
// softmax (3500 cycles), weighted values, is longer than a tile's copy: 4 us a
// tile.  8-bit caches wait for the warps that turn them into fp16, at 4500
// cycles a tile of 128 tokens by 128: 268 MB take 158 us with fp16 queries, 173
// with bf16 ones, whose scaling is on the way from one item to the next.  Heads of
// 192 and 256, 16 + 2 of them over 64 sequences of 4096 tokens, take 110 and 116
// us in bf16 (403 and 537 MB), 156 and 172 us in e4m3.
//
// All hand-overs are mbarriers.  Waits are bounded: one that gave up is
// counted, raises the block's stop flag, on which all others give up too, and
// the block leaves, once what it has under way has had time to land: copies
// and products of warps that were done with their part as much as of those that
// gave up, as the wait that runs out for a late copy is not its own warp's.
#pragma once

#include "ar_tcgen05.cuh"
#include "ar_tree.cuh"

namespace ar {

constexpr unsigned long long kTreeWaitLimitNs = 1000000000ull, kTreeLandNs = 1000000ull;

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
// The same, but never suspended: try_wait may hold the thread for microseconds, which a warp with other things to do has not.
__device__ __forceinline__ bool bar_poll(uint32_t bar, uint32_t parity)
{
    uint32_t done;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
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
    uint32_t valid[4];   // which tokens are in the cache
    int bad;             // whether a value is infinite or NaN, in a tile that some row sees in part only
};

template <typename T_, typename CT_, int DIM_, int NM_>
struct TreeMmaShape {
    using T = T_;
    using CT = CT_;
    using MT = typename std::conditional<sizeof(CT) == 1, __half, CT>::type;  // of the products' operands
    static constexpr int DIM = DIM_, NM = NM_;
    static constexpr bool SMALL = sizeof(CT) == 1, SCALED = SMALL && !std::is_same<T, __half>::value;
    static constexpr bool BF16 = std::is_same<MT, __nv_bfloat16>::value;
    static constexpr int ROWS = 128 * NM, TOKENS = DIM <= 128 ? 128 : 64;
    static constexpr int GROUPS = DIM <= 128 ? 2 : 1;           // softmax warpgroups, each with an O
    static constexpr bool SPLIT = GROUPS == 2 && NM == 1;       // they take alternate tiles
    static_assert(NM <= GROUPS, "a warpgroup for each half of the rows");
    static constexpr int SOFTMAX = 128 * GROUPS, THREADS = SOFTMAX + 128 + 128;
    static constexpr int Q = ROWS * DIM * 2, SLOT = TOKENS * DIM * 2, RAW = SMALL ? TOKENS * DIM : 0;
    static constexpr int MISC = 3 * 1024, ROOM = 232448 - MISC;     // a block's 227 KB
    static constexpr int QS = NM == 1 && DIM == 64 ? 2 : 1;  // heads of 128: another slot of keys or values instead
    static constexpr int RS = !SMALL ? 0 : DIM == 64 ? 8 : 4;
    static constexpr int FIT = (ROOM - QS * Q - RS * RAW) / SLOT, NS = FIT < 10 ? FIT : 10;
    // Score buffers, one a group (or two for its one group): beside two O's tensor memory has no room for more.  Two a group, of
    // half a tile each, gain less than the steps' number costs: 275 against 268 us with 256 rows (539 MB of bf16), 144 against
    // 125 us with up to 128 (537 MB).  Tiles of half the size: 374 against 251 us (286 MB of e4m3).
    static constexpr int BUFFERS = 2;
    static_assert(NS >= 3, "a tile's keys and values, and the next one's keys");
    // Fill f is the keys of tile f / 2, or its values where f is odd.  Keys and values have rings of their own, so that the warps
    // that bring one never wait for those that bring the other.
    static constexpr int KS = NS / 2, VS = NS - KS;
    static __device__ __forceinline__ int slot(int f) { return f & 1 ? KS + (f >> 1) % VS : (f >> 1) % KS; }
    static __device__ __forceinline__ int round(int f) { return f & 1 ? (f >> 1) / VS : (f >> 1) / KS; }
    // The fill before f in its slot.
    static __device__ __forceinline__ int before(int f) { return f - 2 * (f & 1 ? VS : KS); }
    static constexpr int ARRIVALS = 8;  // barriers of fills that need hands: by stage (8-bit), or by tile
    static_assert(RS <= ARRIVALS && (RS == 0 || RS % 4 == 0) && NS <= 16, "a stage is one warp's; a warp has at most four tiles under way");
    static constexpr int TILES = SCALED ? 6 : 8;  // descriptions of tiles
    // Items whose queries' powers of two are kept.  Item i's queries come when the scores of item i - QS are done, and those of a
    // step when the weights of BUFFERS steps before are used: a group's first step of item i - EXPONENTS is behind that.
    static constexpr int EXPONENTS = NM == 2 ? 4 : 6;
    static_assert(EXPONENTS >= QS + 3, "powers are read before they are written over");
    static constexpr int SMEM = QS * Q + NS * SLOT + RS * RAW + MISC;
    // Weights may pass their reference's by 2^AHEAD before it is moved, which costs a pass over O.  fp16 weights are 2^LIFT
    // times as large, so that small ones keep their bits: the largest is 2^15, and the sum holds one of 2^LIFT, so that a weight
    // is off by 2^-25, 2^-36 of that one, where its second number runs out of bits.
    static constexpr float AHEAD = BF16 ? 8.0f : 4.0f, LIFT = BF16 ? 0.0f : 11.0f;
    static constexpr int S_COLUMNS = TOKENS, O_COLUMN = 256;  // score buffers from column 0 on; O of group m at 256 + 128 m
    static_assert(BUFFERS * S_COLUMNS <= O_COLUMN && O_COLUMN + (DIM <= 128 ? GROUPS * 128 : 256) <= 512, "tensor memory");
    static constexpr int BARS = 2 * NS + 2 * QS + 3 * BUFFERS + GROUPS + 2 * TILES + 2 + 2 + ARRIVALS + RS;
    // Step u is half m of the rows of tile t, u = NM t + m.
    static __device__ __forceinline__ int tile_of(int u) { return u / NM; }
    static __device__ __forceinline__ bool first_of_tile(int u) { return u % NM == 0; }
    static __device__ __forceinline__ bool last_of_tile(int u) { return u % NM == NM - 1; }
    static __device__ __forceinline__ int group_of(int u) { return GROUPS == 2 ? u & 1 : 0; }
    static __device__ __forceinline__ int phase_of(int u) { return GROUPS == 2 ? u >> 1 : u; }  // of the group's O
    static __device__ __forceinline__ int buffer_of(int u) { return u % BUFFERS; }
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
    static constexpr uint32_t KV = P::QS * P::Q, RAW = KV + P::NS * P::SLOT, BAR = RAW + P::RS * P::RAW, TILE = BAR + P::BARS * 8,
                              SCALE = TILE + P::TILES * sizeof(TreeTile), JOIN = SCALE + (P::SCALED ? P::EXPONENTS * P::ROWS : 0),
                              SCAN = (JOIN + (P::SPLIT ? 128 * 8 : 0) + 7) / 8 * 8, SENT = SCAN + (P::THREADS / 32 + 2) * 8, END = SENT + 16 + 8;
    __device__ __forceinline__ uint32_t q(int slot) const { return at + slot * P::Q; }
    __device__ __forceinline__ uint32_t kv(int slot) const { return at + KV + slot * P::SLOT; }
    __device__ __forceinline__ char* raw(int stage) const { return base + RAW + stage * P::RAW; }
    __device__ __forceinline__ uint32_t bar(int i) const { return at + BAR + 8 * i; }
    static constexpr int B_Q = 2 * P::NS, B_S = B_Q + 2 * P::QS, B_O = B_S + 3 * P::BUFFERS, B_TILE = B_O + P::GROUPS, B_END = B_TILE + 2 * P::TILES, B_RAW = B_END + 4;
    static_assert(B_RAW + P::ARRIVALS + P::RS == P::BARS, "all barriers");
    __device__ __forceinline__ uint32_t kv_full(int s) const { return bar(s); }
    __device__ __forceinline__ uint32_t kv_empty(int s) const { return bar(P::NS + s); }
    __device__ __forceinline__ uint32_t q_full(int s) const { return bar(B_Q + s); }
    __device__ __forceinline__ uint32_t q_empty(int s) const { return bar(B_Q + P::QS + s); }
    __device__ __forceinline__ uint32_t s_full(int s) const { return bar(B_S + s); }
    __device__ __forceinline__ uint32_t p_ready(int s) const { return bar(B_S + P::BUFFERS + s); }
    __device__ __forceinline__ uint32_t p_used(int s) const { return bar(B_S + 2 * P::BUFFERS + s); }  // weights, by the product
    __device__ __forceinline__ uint32_t o_done(int m) const { return bar(B_O + m); }
    __device__ __forceinline__ uint32_t tile_full(int i) const { return bar(B_TILE + i); }
    __device__ __forceinline__ uint32_t tile_empty(int i) const { return bar(B_TILE + P::TILES + i); }
    __device__ __forceinline__ uint32_t told() const { return bar(B_END); }       // the second group's references are there
    __device__ __forceinline__ uint32_t taken() const { return bar(B_END + 1); }  // its O has been read
    __device__ __forceinline__ uint32_t last(int i) const { return bar(B_END + 2 + i); }
    __device__ __forceinline__ uint32_t arrived(int i) const { return bar(B_RAW + i); }  // copies that need hands
    __device__ __forceinline__ uint32_t raw_empty(int stage) const { return bar(B_RAW + P::ARRIVALS + stage); }
    __device__ __forceinline__ uint32_t sent(int warp) const { return at + SENT + 4 * warp; }  // a copying warp's next tile
    __device__ __forceinline__ TreeTile& tile(int t) const { return reinterpret_cast<TreeTile*>(base + TILE)[t % P::TILES]; }
    __device__ __forceinline__ signed char* exponents(int item) const { return reinterpret_cast<signed char*>(base + SCALE) + item % P::EXPONENTS * P::ROWS; }
    __device__ __forceinline__ float2* join() const { return reinterpret_cast<float2*>(base + JOIN); }
    __device__ __forceinline__ long long* scan() const { return reinterpret_cast<long long*>(base + SCAN); }
    __device__ __forceinline__ uint32_t* tmem() const { return reinterpret_cast<uint32_t*>(base + END - 8); }
    __device__ __forceinline__ int* stop() const { return reinterpret_cast<int*>(base + END - 4); }
    static_assert(TILE % 8 == 0 && JOIN % 8 == 0 && END <= P::SMEM, "shared memory");
};

// One lane of a converged warp.
__device__ __forceinline__ bool elected()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
// ---------------------------------------------------------------------------
// The helping warps.  With tensor copies (help) they bring queries and do what
// is left of fills that need hands.  Without (run: pages that do not fit boxes)
// they copy as well: two take the keys of alternate tiles and two the values,
// each a whole tile's, so that one looks pages up while others' copies queue
// for memory (with a quarter of every tile each, all four did the one and then
// the other: 6000 cycles a tile of 64 KB, half of them for the copies).  16-bit
// elements then go by asynchronous copies straight to the permuted places that
// the tensor core reads, and arrive at the product's barrier by themselves;
// 8-bit ones go to a stage that their own thread turns into fp16, exactly.  A
// warp goes round what it may do next (queries whose slot is free, a fill
// whose slot is free, a fill that has arrived and needs its hands) and waits
// for none while another is possible.  The fence between these writes and the
// tensor core's reads is the issuing warp's: here it would wait for all copies
// on their way.  Pages of 17 tokens, which take this way, are 233 us (bf16
// queries; 238 with fp16 ones) on 268 MB of e4m3, where pages of 64 are 173 (158),
// and 187 us on 537 MB of bf16, where pages of 64 are 125.
// ---------------------------------------------------------------------------
template <typename P>
struct TreeFeed {
    using Cur = TreeCursor<P::ROWS, P::TOKENS>;
    static constexpr int CH = P::DIM * static_cast<int>(sizeof(typename P::CT)) / 16;  // 16-byte chunks of a token
    static constexpr int BLOCKS = P::TOKENS / 32;  // of 32 tokens, one a lane; CH steps of the warp each
    static constexpr int STEPS = CH % 8 == 0 ? 8 : 4;  // at once
    static_assert(CH % STEPS == 0, "whole groups of steps");
    static constexpr int QCH = P::DIM * 2 / 16;
    const TreeArgs& a;
    const TreeSmem<P>& sm;
    volatile int* stop;
    int warp, lane, chunks, qchunks;
    bool values;             // whose the warp is
    uint64_t once, often;    // how long L2 keeps lines
    // The warp's next tile, whose page numbers are on their way.
    int pages[BLOCKS];
    uint64_t at[BLOCKS];     // of the lane's tokens in their pages
    TreeSeq q;
    int b, h, row0, rows, token0, flags;
    bool alone;              // whether no other item reads these tokens
    int tile, passed = 0;    // its number; tiles that the cursor has passed
    int done;                // the warp's oldest tile that may still need its hands
    uint32_t mixeds = 0;     // bits of the last 32 tiles, by number
    uint32_t phases = 0;     // of `arrived`, by number (16-bit)
    Cur item;                // the next item whose queries are wanted, the tile it begins with, and how many were before
    int item_tile = 0, filled = 0;

    __device__ TreeFeed(const TreeArgs& a_, const TreeSmem<P>& sm_, volatile int* stop_, const Cur& cur)
        : a(a_), sm(sm_), stop(stop_), warp((threadIdx.x >> 5) - P::SOFTMAX / 32), lane(threadIdx.x & 31),
          chunks(a_.head_dim * static_cast<int>(sizeof(typename P::CT)) / 16), qchunks(a_.head_dim * 2 / 16), values(warp & 1), tile(warp >> 1),
          done(warp >> 1), item(cur)
    {
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(often));
    }
    static __device__ __forceinline__ void arrive_with_copies(uint32_t bar)
    {
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
    }
    // A row's 16-byte chunk of an operand of `rows` rows.
    static __device__ __forceinline__ uint32_t place(int row, int c, int rows) { return (c >> 3) * (rows * 128) + row * 128 + ((c ^ row) & 7) * 16; }

    // Which of the barriers `arrived` is that of the warp's fill of tile t.
    __device__ __forceinline__ int arrival(int t) const
    {
        return P::SMALL ? (2 * t + (values ? 1 : 0)) % (P::SMALL ? P::RS : 1) : (t & 1) * 4 + (t >> 1 & 3);
    }
    // Whether the fills of a slot are all one warp's.
    static constexpr bool ALONE = P::KS % 2 == 0 && P::VS % 2 == 0;
    // What the warp has sent (16-bit) or handed over (8-bit), for the others.
    __device__ __forceinline__ void tell(int next)
    {
        if (!ALONE && lane == 0)
            asm volatile("st.release.cta.shared::cta.s32 [%0], %1;" ::"r"(sm.sent(warp)), "r"(next) : "memory");
    }
    // Whether fill f's slot is free.  A parity tells two phases apart only, so the fill before it in the slot, where it is another
    // warp's, has to have been sent.
    __device__ __forceinline__ bool free(int f) const
    {
        const int before = P::before(f);
        if (!ALONE && before >= 0) {
            int next;
            asm volatile("ld.acquire.cta.shared::cta.s32 %0, [%1];" : "=r"(next) : "r"(sm.sent((before & 1) + (before >> 1 & 1) * 2)) : "memory");
            if (!__all_sync(~0u, next > before >> 1))
                return false;
        }
        return __all_sync(~0u, bar_poll(sm.kv_empty(P::slot(f)), (P::round(f) & 1) ^ 1));
    }
    // Moves the cursor on to tile `tile`, the warp's next, and asks for its pages.
    __device__ __forceinline__ void look(Cur& cur, const Run& line, int n)
    {
        for (; passed < n; ++passed) {
            const int t = passed;
            const bool begins = cur.tile == 0, ends = cur.tile + 1 == cur.s.tiles, mine = t == tile;
            const int first_token = (cur.s.tile0 + cur.tile) * P::TOKENS;
            if (mine) {
                const bool mixed = tree_mixed(a, cur.q, first_token, P::TOKENS);
                mixeds = (mixeds & ~(1u << (t & 31))) | (mixed ? 1u : 0u) << (t & 31);
                q = cur.q;
                b = cur.b;
                h = cur.h;
                row0 = cur.rt * P::ROWS;
                rows = cur.rows(a);
                token0 = first_token;
                flags = (begins || t == 0 ? kTileFirst : 0) | (ends || t + 1 == n ? kTileLast : 0) | (begins ? kTileBegins : 0) | (ends ? kTileEnds : 0) |
                        (mixed ? kTreeMixed : 0);
                alone = row_blocks<P::ROWS>(a, cur.q) == 1;
#pragma unroll
                for (int k = 0; k < BLOCKS; ++k) {
                    const int token = first_token + 32 * k + lane;
                    pages[k] = -1;
                    if (token >= cur.s.start && token < cur.s.end) {
                        const uint32_t column = __umulhi(2u * token, a.page_magic) >> a.page_shift;
                        pages[k] = a.table[static_cast<uint64_t>(cur.b) * a.table_stride + column];
                        at[k] = static_cast<uint32_t>(token - static_cast<int>(column) * a.page_size) * a.token_stride +
                                static_cast<uint32_t>(cur.h) * a.head_stride;
                    }
                }
            }
            if (begins && n - t < cur.s.tiles && threadIdx.x == P::SOFTMAX)
                leave_job(a, cur, line, t);
            if (t + 1 < n) {
                if (ends)
                    cur.next_item(a);
                else
                    ++cur.tile;
            }
            if (mine) {
                ++passed;
                return;
            }
        }
    }
    // The queries of the next item, where their slot is free.  All copying warps take a part.
    __device__ __forceinline__ bool queries(int n)
    {
        const int s = filled % P::QS;
        if (item_tile >= n || !__all_sync(~0u, bar_poll(sm.q_empty(s), (filled / P::QS & 1) ^ 1)))
            return false;
        const int first = item.q.first, h = item.h, row0 = item.rt * P::ROWS, rows = item.rows(a);
        const uint32_t to = s * P::Q;
        if constexpr (!P::SCALED) {
#pragma unroll 4
            for (int x = warp * 32 + lane; x < P::ROWS * QCH; x += 128) {
                const int row = x / QCH, c = x - row * QCH, i = (row0 + row) / a.group, g = row0 + row - i * a.group;
                const bool read = row < rows && c < qchunks;
                const char* from_q = a.q;
                if (read)
                    from_q += static_cast<uint64_t>(first + i) * a.q_stride + (static_cast<uint64_t>(h) * a.group + g) * a.head_dim * 2 + c * 16;
                cp_async16(sm.at + to + (row >> 7) * (128 * P::DIM * 2) + place(row & 127, c, 128), from_q, read);
            }
            arrive_with_copies(sm.q_full(s));
        } else {
            // bf16 queries on an 8-bit cache: scaled by a power of two a row, so that the largest element becomes 2^14 or more
            // and those down to 2^-28 of it keep all their bits in fp16.
            signed char* const exponents = sm.exponents(filled);
            constexpr int WIDE = QCH <= 8 ? 8 : QCH <= 16 ? 16 : 32, TOGETHER = 32 / WIDE;  // lanes of a row, rows of a step
            const int c = lane % WIDE;
#pragma unroll 4
            for (int row = warp * TOGETHER + lane / WIDE; row < P::ROWS; row += 4 * TOGETHER) {
                const int i = (row0 + row) / a.group, g = row0 + row - i * a.group;
                uint4 w = make_uint4(0, 0, 0, 0);
                if (row < rows && c < qchunks)
                    w = *reinterpret_cast<const uint4*>(a.q + static_cast<uint64_t>(first + i) * a.q_stride +
                                                        (static_cast<uint64_t>(h) * a.group + g) * a.head_dim * 2 + c * 16);
                const float2 f[4] = {Lanes<typename P::T>::two(w.x), Lanes<typename P::T>::two(w.y), Lanes<typename P::T>::two(w.z),
                                     Lanes<typename P::T>::two(w.w)};
                float most = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    most = fmaxf(most, fmaxf(fabsf(f[k].x), fabsf(f[k].y)));
#pragma unroll
                for (int o = WIDE / 2; o > 0; o >>= 1)
                    most = fmaxf(most, __shfl_xor_sync(~0u, most, o));
                const int e = max(static_cast<int>(__float_as_uint(most) >> 23) - 127, -112) - 14;
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                if (c < QCH) {
                    uint4 x;
                    x.x = Lanes<__half>::word(f[0].x * down, f[0].y * down);
                    x.y = Lanes<__half>::word(f[1].x * down, f[1].y * down);
                    x.z = Lanes<__half>::word(f[2].x * down, f[2].y * down);
                    x.w = Lanes<__half>::word(f[3].x * down, f[3].y * down);
                    *reinterpret_cast<uint4*>(sm.base + to + (row >> 7) * (128 * P::DIM * 2) + place(row & 127, c, 128)) = x;
                }
                if (c == 0)
                    exponents[row] = static_cast<signed char>(e);  // -126 .. 114
            }
            bar_arrive(sm.q_full(s));
        }
        ++filled;
        item_tile += item.s.tiles - item.tile;
        if (item_tile < n)
            item.next_item(a);
        return true;
    }
    // Sends tile `tile`'s keys or values on their way, and says what the tile is.
    __device__ __forceinline__ void send(Cur& cur, const Run& line, int n)
    {
        const int t = tile, f = 2 * t + (values ? 1 : 0);
        uint32_t in[BLOCKS], lo[BLOCKS], hi[BLOCKS];
        bool whole = chunks == CH;
#pragma unroll
        for (int k = 0; k < BLOCKS; ++k) {
            const bool ok = pages[k] >= 0 && pages[k] < a.pages;
            const uint64_t off = ok ? static_cast<uint32_t>(pages[k]) * a.page_stride + at[k] : 0;
            lo[k] = static_cast<uint32_t>(off);
            hi[k] = static_cast<uint32_t>(off >> 32);
            in[k] = __ballot_sync(~0u, ok);
            whole = whole && in[k] == ~0u;
        }
        if (!values && lane == 0) {
            TreeTile& x = sm.tile(t);
            x.q = q;
            x.head = h;
            x.row0 = row0;
            x.rows = rows;
            x.token0 = token0;
            x.b = b;
            x.flags = flags;
#pragma unroll
            for (int k = 0; k < BLOCKS; ++k)
                x.valid[k] = in[k];
            bar_arrive(sm.tile_full(t % P::TILES));
        }
        const bool hands = P::SMALL || (values && (flags & kTreeMixed));
        const char* const base = values ? a.v : a.k;
        const uint32_t to = P::SMALL ? smem_addr(sm.raw(f % (P::SMALL ? P::RS : 1))) : sm.kv(P::slot(f));
        const uint64_t policy = alone ? once : often;
        tile += 2;
        look(cur, line, n);
#pragma unroll
        for (int k = 0; k < BLOCKS; ++k) {
#pragma unroll 1
            for (int i0 = 0; i0 < CH; i0 += STEPS) {
                uint32_t x[STEPS], y[STEPS];  // all shuffles, then all copies
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int row = (lane + 32 * (i0 + i)) / CH;
                    x[i] = __shfl_sync(~0u, lo[k], row);
                    y[i] = __shfl_sync(~0u, hi[k], row);
                }
#pragma unroll
                for (int i = 0; i < STEPS; ++i) {
                    const int row = (lane + 32 * (i0 + i)) / CH, c = lane + 32 * (i0 + i) - row * CH;
                    const char* const from = base + (static_cast<uint64_t>(y[i]) << 32 | x[i]) + c * 16;
                    // an 8-bit chunk lies where its own thread finds it
                    const uint32_t dst = P::SMALL ? to + ((k * CH + i0 + i) * 32 + lane) * 16 : to + place(32 * k + row, c, P::TOKENS);
                    if (whole) {
                        cp_async16_all(dst, from, policy);
                    } else {
                        const bool read = (in[k] >> row & 1) != 0 && c < chunks;
                        cp_async16(dst, read ? from : base, read, policy);
                    }
                }
            }
        }
        arrive_with_copies(hands ? sm.arrived(arrival(t)) : sm.kv_full(P::slot(f)));
        if (!P::SMALL)
            tell(tile);
    }
    // 8-bit: turns the warp's oldest fill, once it is here and its slot is free, into fp16 and hands it over.
    __device__ __forceinline__ bool convert()
    {
        const int t = done, f = 2 * t + (values ? 1 : 0);
        constexpr int RS = P::SMALL ? P::RS : 1;
        if (t >= tile || !free(f) || !__all_sync(~0u, bar_poll(sm.arrived(arrival(t)), f / RS & 1)))
            return false;
        done += 2;
        const bool mixed = values && (mixeds >> (t & 31) & 1) != 0;
        char* const to = sm.base + (sm.kv(P::slot(f)) - sm.at);
        const char* const raw = sm.raw(f % RS);
        bool bad = false;
#pragma unroll 1
        for (int i0 = 0; i0 < BLOCKS * CH; i0 += STEPS) {
            uint4 all[STEPS];  // loads before stores, which the compiler may not exchange
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
                all[i] = *reinterpret_cast<const uint4*>(raw + ((i0 + i) * 32 + lane) * 16);
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int row = (lane + 32 * (i0 + i)) / CH, c = lane + 32 * (i0 + i) - row * CH;
                const uint4 w = all[i];
                uint32_t x[8] = {half2_of_e4m3(w.x), half2_of_e4m3(w.x >> 16), half2_of_e4m3(w.y), half2_of_e4m3(w.y >> 16),
                                 half2_of_e4m3(w.z), half2_of_e4m3(w.z >> 16), half2_of_e4m3(w.w), half2_of_e4m3(w.w >> 16)};
                if (mixed) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t y = not_finite<__half>(x[j]);
                        bad = bad || y != 0;
                        x[j] &= ~y;
                    }
                }
                *reinterpret_cast<uint4*>(to + place(row, 2 * c, P::TOKENS)) = make_uint4(x[0], x[1], x[2], x[3]);
                *reinterpret_cast<uint4*>(to + place(row, 2 * c + 1, P::TOKENS)) = make_uint4(x[4], x[5], x[6], x[7]);
            }
        }
        if (mixed) {
            bad = __any_sync(~0u, bad);
            if (lane == 0)
                sm.tile(t).bad = bad;
        }
        bar_arrive(sm.kv_full(P::slot(f)));
        tell(done);
        return true;
    }
    // 16-bit: the values of the warp's oldest tile that rows see in part, once they are here: infinite ones and NaN become 0.
    __device__ __forceinline__ bool look_through()
    {
        while (done < tile && (!values || (mixeds >> (done & 31) & 1) == 0))
            done += 2;
        if (done >= tile)
            return false;
        const int t = done, s = P::slot(2 * t + 1), i = arrival(t);
        if (!__all_sync(~0u, bar_poll(sm.arrived(i), phases >> i & 1)))
            return false;
        phases ^= 1u << i;
        done += 2;
        uint4* const all = reinterpret_cast<uint4*>(sm.base + (sm.kv(s) - sm.at));
        bool bad = false;
#pragma unroll 8
        for (int i = lane; i < P::TOKENS * CH; i += 32) {  // wherever the chunks lie
            const uint4 w = all[i];
            const uint4 x = make_uint4(not_finite<typename P::MT>(w.x), not_finite<typename P::MT>(w.y), not_finite<typename P::MT>(w.z),
                                       not_finite<typename P::MT>(w.w));
            if ((x.x | x.y | x.z | x.w) != 0) {
                bad = true;
                all[i] = make_uint4(w.x & ~x.x, w.y & ~x.y, w.z & ~x.z, w.w & ~x.w);
            }
        }
        bad = __any_sync(~0u, bad);
        if (lane == 0)
            sm.tile(t).bad = bad;
        __syncwarp();
        bar_arrive(sm.kv_full(s));
        return true;
    }
    // Whether the warp's next fill has where to go.
    __device__ __forceinline__ bool room() const
    {
        if (P::SMALL ? (tile - done) / 2 >= P::RS / 4 : !free(2 * tile + (values ? 1 : 0)))
            return false;
        return values || __all_sync(~0u, bar_poll(sm.tile_empty(tile % P::TILES), (tile / P::TILES & 1) ^ 1));
    }
    // Whether nothing has happened for too long, or the block stops.
    __device__ __forceinline__ bool gave_up(unsigned long long& idle_since) const
    {
        unsigned long long now;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(now));
        idle_since = idle_since == 0 ? now : idle_since;
        const bool late = now - idle_since > kTreeWaitLimitNs;
        if (late && *stop == 0) {
            *stop = 1;
            atomicAdd(&g_tree_wait_timeouts, 1u);
        }
        return __any_sync(~0u, late || *stop != 0);
    }
    // 8-bit: a half of a fill, from its stage to its slot.  Bound by the instructions that it issues beside the softmax's: the
    // conversion in five bit operations a pair was 208 us in place of 168, places worked out at every step 168 in place of 157,
    // and stores ordered so that no two lanes meet in a bank 159 (268 MB of e4m3).
    __device__ __forceinline__ void convert_half(TreeTile& x, int f, bool sift)
    {
        constexpr int RS = P::SMALL ? P::RS : 1;
        char* const to = sm.base + (sm.kv(P::slot(f)) - sm.at);
        const char* const raw = sm.raw(f % RS);
        bool bad = false;
        constexpr int HALF = BLOCKS * CH / 2, ONCE = 4;  // steps of the warp, and at once
        static_assert(HALF % ONCE == 0, "whole groups of steps");
        const uint32_t which = warp & 1;
        // Where the rows of a warp's step lie alike in the permutation, in every step, a lane's places are two and a stride.
        constexpr bool ALIKE = 64 % (8 * CH) == 0;
        const uint32_t row0 = (which * 32 + lane) / CH, c0 = (which * 32 + lane) % CH;
        char* const place0 = to + place(row0, 2 * c0, P::TOKENS);
        char* const place1 = to + place(row0, 2 * c0 + 1, P::TOKENS);
        const char* const from = raw + (which * 32 + lane) * 16;
#pragma unroll 1
        for (uint32_t i0 = 0; i0 < HALF; i0 += ONCE) {
            uint4 all[ONCE];
#pragma unroll
            for (int i = 0; i < ONCE; ++i)
                all[i] = *reinterpret_cast<const uint4*>(from + (i0 + i) * 1024);
#pragma unroll
            for (int i = 0; i < ONCE; ++i) {
                const uint32_t at_chunk = ((i0 + i) * 2 + which) * 32 + lane, row = at_chunk / CH, c = at_chunk - row * CH;
                const uint4 w = all[i];
                uint32_t y[8] = {half2_of_e4m3(w.x), half2_of_e4m3(w.x >> 16), half2_of_e4m3(w.y), half2_of_e4m3(w.y >> 16),
                                 half2_of_e4m3(w.z), half2_of_e4m3(w.z >> 16), half2_of_e4m3(w.w), half2_of_e4m3(w.w >> 16)};
                if (sift) {
                    const bool there = x.valid[row >> 5] >> (row & 31) & 1;
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const uint32_t z = not_finite<__half>(y[j]);
                        bad = bad || (there && z != 0);
                        y[j] = there ? y[j] & ~z : 0u;
                    }
                }
                char* const p0 = ALIKE ? place0 + (i0 + i) * (64 / CH * 128) : to + place(row, 2 * c, P::TOKENS);
                char* const p1 = ALIKE ? place1 + (i0 + i) * (64 / CH * 128) : to + place(row, 2 * c + 1, P::TOKENS);
                *reinterpret_cast<uint4*>(p0) = make_uint4(y[0], y[1], y[2], y[3]);
                *reinterpret_cast<uint4*>(p1) = make_uint4(y[4], y[5], y[6], y[7]);
            }
        }
        if (bad)
            x.bad = 1;
    }
    // 16-bit: infinite values and NaN, and whatever lies where no token is, become 0 in a quarter of a tile's values.
    __device__ __forceinline__ void sift_quarter(TreeTile& x, int s)
    {
        bool bad = false;
        char* const to = sm.base + (sm.kv(s) - sm.at);
#pragma unroll 4
        for (int j = warp * 32 + lane; j < P::TOKENS * P::DIM / 8; j += 128) {
            const int row = j / (P::DIM / 8), c = j - row * (P::DIM / 8);
            const bool there = x.valid[row >> 5] >> (row & 31) & 1;
            uint4* const p = reinterpret_cast<uint4*>(to + place(row, c, P::TOKENS));
            const uint4 w = *p;
            const uint4 y = make_uint4(not_finite<typename P::MT>(w.x), not_finite<typename P::MT>(w.y), not_finite<typename P::MT>(w.z),
                                       not_finite<typename P::MT>(w.w));
            const bool found = (y.x | y.y | y.z | y.w) != 0;
            bad = bad || (there && found);
            if (!there)
                *p = make_uint4(0, 0, 0, 0);
            else if (found)
                *p = make_uint4(w.x & ~y.x, w.y & ~y.y, w.z & ~y.z, w.w & ~y.w);
        }
        if (bad)
            x.bad = 1;
    }
    // What tensor copies leave to do: queries, and the fills that need hands: in 8 bits two warps take the keys and two the
    // values, in 16 bits all four the values of tiles that rows see in part.  One loop over the two stages of a tile (its
    // description, then its fill), with queries wherever the next stage has to wait.
    __device__ bool help(int n)
    {
        constexpr int RS = P::SMALL ? P::RS : 1;
        const int kind = P::SMALL ? warp >> 1 : 1;  // 1: values
        uint32_t used = 0;  // phases of `arrived` (16-bit)
        unsigned long long idle_since = 0;
        int t = 0;
        bool described = false;
        while (t < n || item_tile < n) {
            const int f = 2 * t + kind;
            bool can = false;
            if (t < n) {
                if (!described)
                    can = bar_test(sm.tile_full(t % P::TILES), t / P::TILES & 1);
                else if (P::SMALL)
                    can = bar_test(sm.arrived(f % RS), f / RS & 1) && bar_test(sm.kv_empty(P::slot(f)), (P::round(f) & 1) ^ 1);
                else
                    can = bar_test(sm.arrived(t % P::ARRIVALS), used >> (t % P::ARRIVALS) & 1);
            }
            if (!__all_sync(~0u, can)) {
                if (queries(n))
                    idle_since = 0;
                else if (gave_up(idle_since))
                    return false;
                continue;
            }
            idle_since = 0;
            TreeTile& x = sm.tile(t);
            const bool mixed = x.flags & kTreeMixed;
            if (!described && (P::SMALL || mixed)) {
                described = true;
                queries(n);
                continue;
            }
            if (described) {
                if constexpr (P::SMALL) {
                    convert_half(x, f, kind == 1 && mixed);
                } else {
                    used ^= 1u << t % P::ARRIVALS;
                    sift_quarter(x, P::slot(f));
                }
                __syncwarp();
                if (lane == 0) {
                    bar_arrive(sm.kv_full(P::slot(f)));
                    if (P::SMALL)
                        bar_arrive(sm.raw_empty(f % RS));
                }
            }
            __syncwarp();
            if (lane == 0)
                bar_arrive(sm.tile_empty(t % P::TILES));
            ++t;
            described = false;
        }
        return true;
    }
    __device__ bool run(Cur cur, const Run& line, int n)
    {
        look(cur, line, n);
        unsigned long long idle_since = 0;
        for (;;) {
            bool moved;
            if constexpr (P::SMALL)
                moved = convert();
            else
                moved = look_through();
            if (queries(n))
                moved = true;
            if (tile < n && room()) {
                send(cur, line, n);
                moved = true;
            }
            if (moved) {
                idle_since = 0;
                continue;
            }
            if (tile >= n && done >= n && item_tile >= n)
                return true;
            if (gave_up(idle_since))
                return false;
        }
    }
};

// ---------------------------------------------------------------------------
// Tensor copies, where pages are whole groups of eight tokens, in boxes of the
// largest power of two that divides them: a warp for the keys and one for the values look a
// tile's pages up, and each lane asks for a box of up to 64 elements (16-bit;
// all of them in 8 bits) by a page's tokens, which arrives permuted as the
// tensor core reads it.  What it brings for tokens that are not in the cache,
// and the rows of pages that are none, are the helping warps' to clear.  A box
// costs the warp 65 to 110 cycles and a tile some 1900 beside, both less than
// the tile's way from HBM (2900): pages of 8 to 256 tokens are 132 to 125 us on
// 537 MB of bf16.
// ---------------------------------------------------------------------------
template <typename P>
struct TreeBoxes {
    using Cur = TreeCursor<P::ROWS, P::TOKENS>;
    const TreeArgs& a;
    const TreeSmem<P>& sm;
    const TreeMaps& maps;
    volatile int* stop;
    int lane, box, runs, blocks;  // tokens of a box, boxes of tokens and of elements in a tile
    int run_of, block;            // the lane's box
    bool values;                  // whose the warp is
    int shift[P::TOKENS / 32];    // of the boxes that the lane's tokens of each 32 lie in
    uint64_t once, often;
    int page = -1, slot = 0;

    __device__ TreeBoxes(const TreeArgs& a_, const TreeSmem<P>& sm_, const TreeMaps& maps_, volatile int* stop_)
        : a(a_), sm(sm_), maps(maps_), stop(stop_), lane(threadIdx.x & 31), box(a_.boxes), runs(P::TOKENS / box),
          blocks(P::SMALL ? 1 : (a_.head_dim + 63) / 64), run_of(lane / blocks), block(lane - run_of * blocks),
          values((threadIdx.x >> 5) == P::THREADS / 32 - 1)
    {
        asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(once));
        asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(often));
#pragma unroll
        for (int k = 0; k < P::TOKENS / 32; ++k)
            shift[k] = (32 * k + lane) / box * blocks;
    }
    // The page of the lane's box; there are 32 at most (16 by 2 of 8 tokens, 8 by 4).
    __device__ __forceinline__ void look_up(const Cur& cur)
    {
        const int token = (cur.s.tile0 + cur.tile) * P::TOKENS + run_of * box;
        page = -1;
        if (run_of < runs && token < cur.s.end && token + box > cur.s.start) {
            const uint32_t column = __umulhi(2u * token, a.page_magic) >> a.page_shift;
            slot = token - static_cast<int>(column) * a.page_size;
            page = a.table[static_cast<uint64_t>(cur.b) * a.table_stride + column];
        }
    }
    __device__ __forceinline__ void copy(uint32_t to, const void* map, int x, int token, int head, int at_page, uint32_t bar, uint64_t policy)
    {
        const int c1 = a.token_first ? token : head, c2 = a.token_first ? head : token;
        asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(to),
                     "l"(map), "r"(x), "r"(c1), "r"(c2), "r"(at_page), "r"(bar), "l"(policy)
                     : "memory");
    }
    __device__ bool run(Cur cur, const Run& line, int n)
    {
        look_up(cur);
        for (int t = 0; t < n; ++t) {
            const bool begins = cur.tile == 0, ends = cur.tile + 1 == cur.s.tiles;
            const int token0 = (cur.s.tile0 + cur.tile) * P::TOKENS, head = cur.h;
            const int good = page >= 0 && page < a.pages ? page : -1, at_slot = slot;
            const uint32_t there = __ballot_sync(~0u, good >= 0);  // boxes
            uint32_t valid[P::TOKENS / 32];
            bool whole = true;
#pragma unroll
            for (int k = 0; k < P::TOKENS / 32; ++k) {
                const int token = token0 + 32 * k + lane;
                valid[k] = __ballot_sync(~0u, token >= cur.s.start && token < cur.s.end && (there >> shift[k] & 1) != 0);
                whole = whole && valid[k] == ~0u;
            }
            const bool mixed = !whole || tree_mixed(a, cur.q, token0, P::TOKENS);
            if (!values) {
                if (!bar_wait(sm.tile_empty(t % P::TILES), (t / P::TILES & 1) ^ 1, stop))
                    return false;
                if (lane == 0) {
                    TreeTile& x = sm.tile(t);
                    x.q = cur.q;
                    x.head = head;
                    x.row0 = cur.rt * P::ROWS;
                    x.rows = cur.rows(a);
                    x.token0 = token0;
                    x.b = cur.b;
                    x.bad = 0;
                    x.flags = (begins || t == 0 ? kTileFirst : 0) | (ends || t + 1 == n ? kTileLast : 0) | (begins ? kTileBegins : 0) | (ends ? kTileEnds : 0) |
                              (mixed ? kTreeMixed : 0);
#pragma unroll
                    for (int k = 0; k < P::TOKENS / 32; ++k)
                        x.valid[k] = valid[k];
                    if (begins && n - t < cur.s.tiles)
                        leave_job(a, cur, line, t);
                    bar_arrive(sm.tile_full(t % P::TILES));
                }
                __syncwarp();
            }
            const uint64_t policy = row_blocks<P::ROWS>(a, cur.q) == 1 ? once : often;
            if (t + 1 < n) {
                if (ends)
                    cur.next_item(a);
                else
                    ++cur.tile;
                look_up(cur);
            }
            {
                const int f = 2 * t + (values ? 1 : 0);
                uint32_t to, bar;
                bool hands = P::SMALL;
                if constexpr (P::SMALL) {
                    constexpr int RS = P::SMALL ? P::RS : 1;
                    if (!bar_wait(sm.raw_empty(f % RS), (f / RS & 1) ^ 1, stop))
                        return false;
                    to = smem_addr(sm.raw(f % RS));
                    bar = sm.arrived(f % RS);
                } else {
                    if (!bar_wait(sm.kv_empty(P::slot(f)), (P::round(f) & 1) ^ 1, stop))
                        return false;
                    to = sm.kv(P::slot(f));
                    hands = (f & 1) != 0 && mixed;
                    bar = hands ? sm.arrived(t % P::ARRIVALS) : sm.kv_full(P::slot(f));
                }
                if (elected()) {
                    const uint32_t bytes = __popc(there) * box * (P::SMALL ? P::DIM : 128);
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
                    if (!hands)  // in the place of the helping warps
                        asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], 3;" ::"r"(bar) : "memory");
                }
                __syncwarp();
                if (good >= 0)  // each lane asks for its box
                    copy(to + (P::SMALL ? run_of * box * P::DIM : block * (P::TOKENS * 128) + run_of * box * 128), f & 1 ? &maps.v : &maps.k, 64 * block,
                         at_slot, head, good, bar, policy);
                __syncwarp();
            }
        }
        return true;
    }
};

// ---------------------------------------------------------------------------
// The products, a warp for the scores and one for the weighted values: a group
// of eight or sixteen costs its warp some 400 cycles of waits and barriers
// beside their own time, which one warp for both spent between them (8100
// cycles a tile of 128 tokens and 256 rows; the products take 3700).  All lanes
// go through the loops and one issues.
// ---------------------------------------------------------------------------
template <typename P>
__device__ bool tree_scores(const TreeArgs& a, const TreeSmem<P>& sm, uint32_t tmem, int n, volatile int* stop)
{
    const int ksteps = (a.head_dim + 15) / 16;
    const uint32_t desc = product_desc(P::BF16, P::TOKENS, false);
    int items = 0;  // whose queries have been waited for
    bool last = false;
    for (int u = 0; u < n * P::NM; ++u) {
        const int t = P::tile_of(u), s = P::slot(2 * t);
        if (P::first_of_tile(u)) {
            if (!bar_wait(sm.tile_full(t % P::TILES), t / P::TILES & 1, stop))
                return false;
            const int flags = __shfl_sync(~0u, sm.tile(t).flags, 0);
            last = flags & kTileLast;
            if (flags & kTileFirst) {
                if (!bar_wait(sm.q_full(items % P::QS), items / P::QS & 1, stop))
                    return false;
                ++items;
            }
            if (!bar_wait(sm.kv_full(s), P::round(2 * t) & 1, stop))
                return false;
            fence_async_proxy();  // between the copying warps' writes, which the barrier has shown, and the product's reads
        }
        // The buffer holds the weights of the step that had it before until their product is done.
        if (!bar_wait(sm.p_used(P::buffer_of(u)), (u / P::BUFFERS & 1) ^ 1, stop))
            return false;
        tcgen05_after_sync();
        const uint64_t q = operand_desc(sm.q((items - 1) % P::QS) + u % P::NM * (128 * P::DIM * 2), 16, 1024),
                       k = operand_desc(sm.kv(s), 16, 1024);
        const uint32_t d = tmem + P::buffer_of(u) * P::S_COLUMNS;
        const bool one = elected();
        // 32 bytes on, then the next 64 elements' block; addresses count 16 bytes
#pragma unroll
        for (int j = 0; j < P::DIM / 16; ++j)
            if (j < ksteps)
                mma_shared(d, q + (j >> 2) * (128 * 128 / 16) + (j & 3) * 2, k + (j >> 2) * (P::TOKENS * 128 / 16) + (j & 3) * 2, desc, j > 0, one);
        tcgen05_commit(sm.s_full(P::buffer_of(u)), one);
        if (P::SCALED && one)  // the queries' powers of two, which the wait for the queries has shown this warp, to the softmax too
            bar_arrive(sm.s_full(P::buffer_of(u)));
        if (P::last_of_tile(u)) {
            tcgen05_commit(sm.kv_empty(s), one);
            if (last)
                tcgen05_commit(sm.q_empty((items - 1) % P::QS), one);
        }
        __syncwarp();
    }
    return true;
}

template <typename P>
__device__ bool tree_values(const TreeArgs& a, const TreeSmem<P>& sm, uint32_t tmem, int n, volatile int* stop)
{
    const uint32_t desc = product_desc(P::BF16, (a.head_dim + 15) / 16 * 16, true);
    bool first = false, second = false;  // whether the tile is the first of the block's part of an item, or the one after it
    for (int u = 0; u < n * P::NM; ++u) {
        const int t = P::tile_of(u), f = 2 * t + 1, s = P::slot(f);
        if (P::first_of_tile(u)) {
            if (!bar_wait(sm.tile_full(t % P::TILES), t / P::TILES & 1, stop))
                return false;
            second = first;
            first = __shfl_sync(~0u, sm.tile(t).flags, 0) & kTileFirst;
            if (elected())
                bar_arrive(sm.tile_empty(t % P::TILES));  // the softmax may be done with it long before this warp looks
            if (!bar_wait(sm.kv_full(s), P::round(f) & 1, stop))
                return false;
            fence_async_proxy();
        }
        // Of the group's O: with alternate tiles, two of an item are first ones.
        const bool begins = first || (P::SPLIT && second);
        if (!bar_wait(sm.p_ready(P::buffer_of(u)), u / P::BUFFERS & 1, stop))
            return false;
        tcgen05_after_sync();
        const uint32_t p = tmem + P::buffer_of(u) * P::S_COLUMNS, o = tmem + P::O_COLUMN + P::group_of(u) * 128;
        const uint64_t v = operand_desc(sm.kv(s), P::TOKENS * 128, 1024);
        const bool one = elected();
#pragma unroll
        for (int j = 0; j < P::TOKENS / 16; ++j) {
            const uint32_t w = p + (j >> 1) * 32 + (j & 1) * 8;  // of 32 tokens 16 columns of weights, then 16 of what they leave
            mma_tensor(o, w, v + j * (2048 / 16), desc, !(begins && j == 0), one);
            mma_tensor(o, w + 16, v + j * (2048 / 16), desc, true, one);
        }
        tcgen05_commit(sm.o_done(P::group_of(u)), one);  // first: who sees the weights used takes this for done
        tcgen05_commit(sm.p_used(P::buffer_of(u)), one);
        if (P::last_of_tile(u))
            tcgen05_commit(sm.kv_empty(s), one);
        __syncwarp();
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
    int m, row, lane;    // group, row of the item
    uint32_t lanes;      // the warp's lanes in an address of tensor memory
    uint32_t o;          // the group's O
    int joins = 0;       // items whose two O's were joined
    bool awaits = false; // the second group's O of the last of them may not have been read yet
    float factor = 0.0f, reference = -INFINITY, total = 0.0f;
    TreeRow sees;

    __device__ TreeSoft(const TreeArgs& a_, const TreeSmem<P>& sm_, uint32_t tmem, volatile int* stop_) : a(a_), sm(sm_), stop(stop_)
    {
        const int warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        m = warp >> 2;
        row = P::SPLIT ? threadIdx.x & 127 : threadIdx.x;
        lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        o = tmem + lanes + P::O_COLUMN + m * 128;
    }
    // Which of 32 tokens of a tile the row sees.
    __device__ __forceinline__ uint32_t seen(const TreeTile& tile, int c) const
    {
        const uint32_t word = tile.valid[c];
        return tile.flags & kTreeMixed ? word & sees.sees(tile.token0 + 32 * c) : word;
    }
    // Weights of a tile whose scores lie at `s`.  PART: not every row sees every token.  CAP: with softcap.  One loop over
    // groups of 32 tokens, not unrolled: the four warps' instructions have to stay in the cache.
    template <bool PART, bool CAP>
    __device__ __forceinline__ bool weights(const TreeTile& tile, uint32_t s, bool first, int u)
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
            if (!bar_wait(sm.o_done(m), P::phase_of(u) - 1 & 1, stop))
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
    __device__ __forceinline__ bool weights(const TreeTile& tile, uint32_t s, bool first, int u, bool part)
    {
        if (a.softcap > 0.0f)
            return weights<true, true>(tile, s, first, u);
        return part ? weights<true, false>(tile, s, first, u) : weights<false, false>(tile, s, first, u);
    }
    // Waits for step u's product with the values; the group's one before was waited for already.
    __device__ __forceinline__ bool weighted(int u)
    {
        if (!bar_wait(sm.o_done(m), P::phase_of(u) & 1, stop))
            return false;
        tcgen05_after_sync();
        return true;
    }
    // Values that are infinite or NaN, in a tile that rows see in part: the product took 0 for them, and the rows that see
    // them get them here, out of the cache once more.
    __device__ __forceinline__ bool poison(const TreeTile& tile, int u, bool valid)
    {
        if (!weighted(u))
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
                for (uint32_t word = tile.valid[c] & sees.sees(tile.token0 + 32 * c); word != 0; word &= word - 1) {
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
    // Before the group's O is written anew, or its references: that the first group has read them.
    __device__ __forceinline__ bool joined()
    {
        if (P::SPLIT && awaits) {
            if (!bar_wait(sm.taken(), joins - 1 & 1, stop))
                return false;
            awaits = false;
        }
        return true;
    }
    // The end of the block's part of an item: the result, or the part.  u: the group's last step of it, -1: it had none.
    __device__ __forceinline__ bool finish(const TreeTile& tile, int u, bool began, bool any, bool valid)
    {
        if (u >= 0 && !weighted(u))
            return false;
        float mine = 1.0f, others = 0.0f;  // what the two O's are multiplied by
        bool both = false;                 // whether the other one has a tile
        const uint32_t other = o + 128;
        if constexpr (P::SPLIT) {
            if (m == 1) {
                if (!joined())
                    return false;
                sm.join()[row] = make_float2(reference, u >= 0 ? total : -1.0f);
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0)
                    bar_arrive(sm.told());
                ++joins;
                awaits = true;
                return true;
            }
            if (!bar_wait(sm.told(), joins++ & 1, stop))
                return false;
            tcgen05_after_sync();
            const float2 x = sm.join()[row];
            both = !(x.y < 0.0f);
            if (both) {  // without a tile of the first group's own its reference is minus infinity, its sum 0
                const float best = fmaxf(reference, x.x), base = base_of(best);
                mine = exp2_fast(reference - base);
                others = exp2_fast(x.x - base);
                total = total * mine + x.y * others;
                reference = best;
            }
        }
        if (any) {
            const bool whole = began && (tile.flags & kTileEnds);
            const uint64_t out = valid ? tree_out_row(a, tile.q.first, tile.head, tile.row0 + row) : 0;
            float* const part = a.part + slot_of(static_cast<int>(blockIdx.x), began) * a.slot_floats;
            const float f = !whole ? 1.0f : total == 0.0f ? 0.0f : a.v_scale / total;
#pragma unroll 1
            for (int c = 0; c < a.head_dim; c += 32) {
                uint32_t x[32];
                tmem_load32(o + c, x);
                tcgen05_wait_load();
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    x[i] = u < 0 ? 0u : __float_as_uint(__uint_as_float(x[i]) * mine);
                if (both) {
                    uint32_t y[32];
                    tmem_load32(other + c, y);
                    tcgen05_wait_load();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        x[i] = __float_as_uint(fmaf(__uint_as_float(y[i]), others, __uint_as_float(x[i])));
                }
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
        }
        if constexpr (P::SPLIT) {
            tcgen05_before_sync();
            __syncwarp();
            if (lane == 0)
                bar_arrive(sm.taken());
        }
        return true;
    }
    __device__ bool run(uint32_t tmem, int n)
    {
        bool began = false, valid = false, any = false;
        int items = 0, own = -1;  // the group's last step of the item
        for (int t = 0; t < n; ++t) {
            if (!bar_wait(sm.tile_full(t % P::TILES), t / P::TILES & 1, stop))
                return false;
            const TreeTile& tile = sm.tile(t);
            const int flags = tile.flags;
            if (flags & kTileFirst) {
                began = flags & kTileBegins;
                valid = row < tile.rows;
                any = __any_sync(~0u, valid);
                sees.make(a, tile.q, (tile.row0 + (valid ? row : 0)) / a.group);
                reference = -INFINITY;
                total = 0.0f;
                own = -1;
                factor = a.scale2;
                ++items;
            }
            if (!P::SPLIT || (t & 1) == m) {
                const int u = P::NM == 2 ? 2 * t + m : t;
                if (!bar_wait(sm.s_full(P::buffer_of(u)), u / P::BUFFERS & 1, stop))
                    return false;
                tcgen05_after_sync();
                if (P::SCALED && own < 0)  // finite: an infinite factor would make the scores of keys that are 0 NaN
                    factor = fmaxf(fminf(ldexpf(a.scale2, sm.exponents(items - 1)[row]), FLT_MAX), -FLT_MAX);
                if (any) {
                    bool part = flags & kTreeMixed;
#pragma unroll
                    for (int w = 0; w < P::TOKENS / 32; ++w)
                        part = part || tile.valid[w] != ~0u;
                    const uint32_t s = tmem + lanes + P::buffer_of(u) * P::S_COLUMNS;
                    if (!weights(tile, s, own < 0, u, part))
                        return false;
                }
                bool bad = false;
                if (flags & kTreeMixed) {  // the values have to be there first; once the weights are, their slot may be filled anew
                    const int f = 2 * t + 1;
                    if (!bar_wait(sm.kv_full(P::slot(f)), P::round(f) & 1, stop))
                        return false;
                    bad = any && *const_cast<const volatile int*>(&tile.bad) != 0;
                }
                // A parity tells two phases apart only: where this step's product is waited for, the group's last one has to be
                // seen done before it can be.  (The one before that was, when this step's scores were begun.)
                if ((bad || (flags & kTileLast)) && P::phase_of(u) > 0 && !bar_wait(sm.o_done(m), P::phase_of(u) - 1 & 1, stop))
                    return false;
                if (!joined())
                    return false;
                tcgen05_before_sync();
                __syncwarp();
                if (lane == 0 && u + 1 != a.stall)
                    bar_arrive(sm.p_ready(P::buffer_of(u)));
                own = u;
                if (bad && !poison(tile, u, valid))
                    return false;
            }
            if ((flags & kTileLast) && !finish(tile, own, began, any, valid))
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
k_tree_mma(const TreeArgs a, const __grid_constant__ TreeMaps maps)
{
    extern __shared__ __align__(1024) char dynamic[];  // all of a block's shared memory: it begins aligned
    pdl_enter();
    const TreeSmem<P> sm(dynamic);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int COPY = P::SOFTMAX / 32, ISSUE = COPY + 4, BOXES = ISSUE + 2;
    volatile int* const stop = sm.stop();
    if (warp == ISSUE)
        tmem_alloc(smem_addr(sm.tmem()), 512);
    if (threadIdx.x == 0) {
        *stop = 0;
        for (int i = 0; i < P::NS; ++i) {
            bar_init(sm.kv_full(i), a.boxes ? (P::SMALL ? 2 : 4) : 32);  // the helping warps, or a copying warp's threads
            bar_init(sm.kv_empty(i), 1);
        }
        for (int i = 0; i < P::QS; ++i) {
            bar_init(sm.q_full(i), 128);
            bar_init(sm.q_empty(i), 1);
        }
        for (int i = 0; i < P::BUFFERS; ++i) {
            bar_init(sm.s_full(i), P::SCALED ? 2 : 1);
            bar_init(sm.p_ready(i), 4);
            bar_init(sm.p_used(i), 1);
        }
        for (int i = 0; i < P::GROUPS; ++i)
            bar_init(sm.o_done(i), 1);
        for (int i = 0; i < P::TILES; ++i) {
            bar_init(sm.tile_full(i), 1);
            bar_init(sm.tile_empty(i), P::SOFTMAX / 32 + 1 + (a.boxes ? 4 : 0));
        }
        bar_init(sm.told(), 4);
        bar_init(sm.taken(), 4);
        bar_init(sm.last(0), 1);
        bar_init(sm.last(1), 1);
        for (int i = 0; i < P::ARRIVALS; ++i)
            bar_init(sm.arrived(i), a.boxes ? 1 : 32);
        for (int i = 0; i < P::RS; ++i)
            bar_init(sm.raw_empty(i), 2);
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<int*>(dynamic + TreeSmem<P>::SENT + 4 * i) = i >> 1;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        a.jobs[blockIdx.x].rows = 0;
    }
    tcgen05_before_sync();
    __syncthreads();
    tcgen05_after_sync();
    const uint32_t tmem = __shfl_sync(~0u, *sm.tmem(), 0);
    TreeCursor<P::ROWS, P::TOKENS> cur;
    const Run line = tree_run<P::ROWS, P::TOKENS, P::THREADS>(a, cur, sm.scan());  // the job's 0 is written before: it contains a barrier
    const int n = static_cast<int>(min(line.n, static_cast<long long>(INT_MAX / 4)));
    if (n > 0) {
        if (warp >= BOXES) {
            if (a.boxes) {
                TreeBoxes<P> boxes(a, sm, maps, stop);
                boxes.run(cur, line, n);
            }
            __syncwarp();
        } else if (warp >= ISSUE) {
            const bool good = warp == ISSUE ? tree_scores<P>(a, sm, tmem, n, stop) : tree_values<P>(a, sm, tmem, n, stop);
            if (!good && lane == 0) {
                // Stopped: the products under way end before shared and tensor memory are given back.
                const uint32_t bar = sm.last(warp - ISSUE);
                tcgen05_commit(bar);
                unsigned long long t0, t;
                asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
                do
                    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
                while (!bar_test(bar, 0) && t - t0 < kTreeWaitLimitNs);
            }
            __syncwarp();
        } else if (warp >= COPY) {
            TreeFeed<P> feed(a, sm, stop, cur);
            if (a.boxes)
                feed.help(n);
            else
                feed.run(cur, line, n);
            asm volatile("cp.async.wait_all;" ::: "memory");  // nothing is left to wait for unless the block stops
            __syncwarp();
        } else {
            TreeSoft<P> soft(a, sm, tmem, stop);
            soft.run(tmem, n);
            __syncwarp();
        }
    }
    tcgen05_before_sync();
    __syncthreads();
    if (*stop != 0) {  // tensor copies and products under way, whosever they are, land within microseconds
        unsigned long long t0, t;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        do
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
        while (t - t0 < kTreeLandNs);
    }
    __syncwarp();
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
cudaError_t launch_tree_mma(const TreeArgs& a, const TreeMaps& maps, const TreeShape& shape, int most, int sms, cudaStream_t s)
{
    const int blocks = most < sms ? most : sms;
    if constexpr (DIM <= 128) {
        if (shape.rows == 256) {
            using P = TreeMmaShape<T, CT, DIM, 2>;
            return launch_tree_kernel<T>(k_tree_mma<P>, a, P::THREADS, P::SMEM, blocks, sms, s, maps);
        }
    }
    using P = TreeMmaShape<T, CT, DIM, 1>;
    return launch_tree_kernel<T>(k_tree_mma<P>, a, P::THREADS, P::SMEM, blocks, sms, s, maps);
}

template <typename T, typename CT>
cudaError_t launch_tree(const TreeArgs& a, const TreeMaps& maps, const TreeShape& shape, int most, int sms, cudaStream_t s)
{
    return a.head_dim <= 64    ? launch_tree_mma<T, CT, 64>(a, maps, shape, most, sms, s)
           : a.head_dim <= 128 ? launch_tree_mma<T, CT, 128>(a, maps, shape, most, sms, s)
           : a.head_dim <= 192 ? launch_tree_mma<T, CT, 192>(a, maps, shape, most, sms, s)
                               : launch_tree_mma<T, CT, 256>(a, maps, shape, most, sms, s);
}

}  // namespace ar
