// ar_pages.cu -- moving cached tokens and pages of the paged key-value cache,
// all layers in one launch: compacting the drafted tokens that were kept, and
// copying pages.
#include <climits>

#include "ar_cache.h"
#include "ar_kernels.cuh"
#include "ar_launch_k.cuh"

namespace ar {

constexpr int kMoveThreads = 256;

template <int BYTES>
struct MoveUnit;
template <>
struct MoveUnit<16> { using type = uint4; };
template <>
struct MoveUnit<8> { using type = uint2; };
template <>
struct MoveUnit<4> { using type = uint32_t; };
template <>
struct MoveUnit<2> { using type = uint16_t; };
template <>
struct MoveUnit<1> { using type = uint8_t; };

// ---------------------------------------------------------------------------
// Copying pages.  A block takes one pair's segment of a page in one buffer (a
// layer's keys or values): PER units a thread, all loads at once.  Whether the pair is
// made it finds by one pass over all pairs, 8 bytes each.  Large pages and few pairs
// hide that behind the other blocks' copies and are bound by HBM: 2000 pages of 32 KB
// in 4 layers, 1.05 GB read and written, take 145 us, 7.2 TB/s.  Thousands of small
// pages are bound by the passes, whose bytes grow with the pairs squared: 4 KB in 8
// layers take 309 us for 4000 pairs, four times their bytes' time, and 2.99 ms for
// 16000, ten times.  8 pages of 4 KB in 16 layers are a launch, 4.5 us.
// ---------------------------------------------------------------------------
template <int BYTES, int PER>
__global__ void __launch_bounds__(kMoveThreads)
k_kv_copy_pages(const CopyArgs a)
{
    using U = typename MoveUnit<BYTES>::type;
    pdl_enter();
    const int pair = static_cast<int>(blockIdx.x / a.segments);
    const uint32_t segment = blockIdx.x - pair * a.segments;
    const int src = a.src[pair], dst = a.dst[pair];
    const auto moves = [&](int s, int d) {
        return s != d && static_cast<unsigned>(s) < static_cast<unsigned>(a.pages) && static_cast<unsigned>(d) < static_cast<unsigned>(a.pages);
    };
    if (!moves(src, dst))
        return;
    bool clash = false;
#pragma unroll 8
    for (int i = threadIdx.x; i < a.pairs; i += kMoveThreads) {
        const int s = a.src[i], d = a.dst[i];
        clash = clash || (moves(s, d) && (d == src || (d == dst && i > pair)));
    }
    if (__syncthreads_or(clash))
        return;
    char* const base = blockIdx.y & 1 ? a.to.odd[blockIdx.y >> 1] : a.to.even[blockIdx.y >> 1];
    const char* const from = base + static_cast<uint64_t>(src) * a.page_stride;
    char* const to = base + static_cast<uint64_t>(dst) * a.page_stride;
    U v[PER];
    uint64_t at[PER];
    const uint64_t first = static_cast<uint64_t>(segment) * (kMoveThreads * PER) + threadIdx.x;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const uint64_t unit = first + i * kMoveThreads;
        at[i] = unit < a.units ? unit * BYTES : ~0ull;
        if (a.inner != a.units && at[i] != ~0ull) {
            const uint32_t row = static_cast<uint32_t>(unit) / a.inner, outer = row / a.mid;
            at[i] = (static_cast<uint32_t>(unit) - row * a.inner) * static_cast<uint64_t>(BYTES) + (row - outer * a.mid) * a.mid_stride +
                    outer * a.outer_stride;
        }
        if (at[i] != ~0ull)
            v[i] = *reinterpret_cast<const U*>(from + at[i]);
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (at[i] != ~0ull)
            *reinterpret_cast<U*>(to + at[i]) = v[i];
}

template <int BYTES>
static cudaError_t launch_copy_unit(const CopyArgs& args, int buffers, cudaStream_t s)
{
    CopyArgs a = args;
    const auto segments_of = [&](int per) { return (a.units + static_cast<uint64_t>(kMoveThreads) * per - 1) / (static_cast<uint64_t>(kMoveThreads) * per); };
    // Eight units a thread where that still leaves every SM eight blocks, else one, for more blocks.
    const bool many = segments_of(8) * a.pairs * buffers >= 152 * 8;
    const uint64_t segments = segments_of(many ? 8 : 1);
    if (segments * a.pairs > static_cast<uint64_t>(INT_MAX))
        return cudaErrorInvalidConfiguration;
    a.segments = static_cast<uint32_t>(segments);
    const dim3 grid(static_cast<unsigned>(segments * a.pairs), buffers);
    return many ? launch_k(k_kv_copy_pages<BYTES, 8>, grid, dim3(kMoveThreads), 0, s, a)
                : launch_k(k_kv_copy_pages<BYTES, 1>, grid, dim3(kMoveThreads), 0, s, a);
}

cudaError_t launch_copy_pages(const CopyArgs& a, int buffers, int unit, cudaStream_t s)
{
    switch (unit) {
    case 16: return launch_copy_unit<16>(a, buffers, s);
    case 8: return launch_copy_unit<8>(a, buffers, s);
    case 4: return launch_copy_unit<4>(a, buffers, s);
    case 2: return launch_copy_unit<2>(a, buffers, s);
    default: return launch_copy_unit<1>(a, buffers, s);
    }
}

// ---------------------------------------------------------------------------
// Compacting.  Kept token j moves from C + kept[j] to C + j.  As kept is
// ascending, a token's new place was the place of an earlier one or of none,
// so taking the tokens in order never overwrites one that is still to move.  A
// thread owns one unit (16 bytes of one head, of one layer's keys or values)
// of all of a sequence's tokens and takes them in order, AHEAD loads at once
// before their stores: no two threads touch the same bytes, as each buffer is
// listed once, and no barrier is needed between moves.  Bound by HBM for large batches, by the chain of loads
// list, length, page, token for small ones (13.1 and 5.1 us; the chain, with
// its barriers, is 4 us of both).
// ---------------------------------------------------------------------------
template <int BYTES>
__global__ void __launch_bounds__(kMoveThreads)
k_kv_compact(const CompactArgs a)
{
    using U = typename MoveUnit<BYTES>::type;
    constexpr int AHEAD = 8;
    constexpr int ROUND = 128;  // tokens whose places are in shared memory at once
    static_assert(ROUND % AHEAD == 0 && ROUND <= kMoveThreads, "whole groups, a thread a token");
    __shared__ int64_t s_from[ROUND], s_to[ROUND];  // byte offsets; s_to -1: not moved
    __shared__ int s_count;
    pdl_enter();
    const int b = static_cast<int>(blockIdx.x), tid = static_cast<int>(threadIdx.x);
    const int length = a.lengths[b];
    const int64_t n = a.seq_start != nullptr ? static_cast<int64_t>(a.seq_start[b + 1]) - a.seq_start[b] : a.drafted;
    const int64_t context = static_cast<int64_t>(length) - n;
    const int* const kept = a.kept + b * a.kept_stride;
    const bool idle = n <= 0 || context < 0;
    // How many are kept: up to the first entry that is not above the one before and below n.
    if (tid == 0)
        s_count = idle ? 0 : a.most_kept;
    __syncthreads();
    if (!idle) {
        for (int j = tid; j < a.most_kept; j += kMoveThreads) {
            const int x = kept[j], before = j > 0 ? kept[j - 1] : -1;
            if (x <= before || x >= n)
                atomicMin(&s_count, j);
        }
    }
    __syncthreads();
    const int count = s_count;
    if (blockIdx.y == 0 && tid == 0)
        a.new_lengths[b] = idle ? length : static_cast<int>(context) + count;
    const uint32_t unit = blockIdx.y * kMoveThreads + tid;
    char* base = nullptr;
    if (unit < a.units) {
        const uint32_t part = unit / a.head_units, in = unit - part * a.head_units, head = in / a.inner;
        base = (part & 1 ? a.to.odd[part >> 1] : a.to.even[part >> 1]) + head * a.head_stride + (in - head * a.inner) * static_cast<uint64_t>(BYTES);
    }
    const int* const table = a.table + static_cast<uint64_t>(b) * a.table_stride;
    const auto place = [&](int64_t token) -> int64_t {
        if (static_cast<uint64_t>(token) >= a.capacity)
            return -1;
        const uint32_t column = static_cast<uint32_t>(token) / static_cast<uint32_t>(a.page_size);
        const int page = table[column];
        if (page < 0 || page >= a.pages)
            return -1;
        return static_cast<int64_t>(static_cast<uint64_t>(page) * a.page_stride +
                                    (static_cast<uint32_t>(token) - column * a.page_size) * a.token_stride);
    };
    for (int j0 = 0; j0 < count; j0 += ROUND) {
        if (tid < ROUND) {
            const int j = j0 + tid;
            int64_t from = -1, to = -1;
            if (j < count && kept[j] != j) {
                from = place(context + kept[j]);
                to = place(context + j);
            }
            s_from[tid] = from;
            s_to[tid] = from < 0 ? -1 : to;
        }
        __syncthreads();
        const int round = min(ROUND, count - j0);
        if (base != nullptr) {
            for (int j = 0; j < round; j += AHEAD) {
                U v[AHEAD];
                int64_t to[AHEAD];
#pragma unroll
                for (int i = 0; i < AHEAD; ++i) {
                    to[i] = s_to[j + i];
                    if (to[i] >= 0)
                        v[i] = *reinterpret_cast<const U*>(base + s_from[j + i]);
                }
#pragma unroll
                for (int i = 0; i < AHEAD; ++i)
                    if (to[i] >= 0)
                        *reinterpret_cast<U*>(base + to[i]) = v[i];
            }
        }
        __syncthreads();
    }
}

cudaError_t launch_compact(const CompactArgs& a, int unit, cudaStream_t s)
{
    const uint32_t columns = (a.units + kMoveThreads - 1) / kMoveThreads;
    if (columns > 65535)
        return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(a.batch), columns > 0 ? columns : 1), block(kMoveThreads);
    switch (unit) {
    case 16: return launch_k(k_kv_compact<16>, grid, block, 0, s, a);
    case 8: return launch_k(k_kv_compact<8>, grid, block, 0, s, a);
    case 4: return launch_k(k_kv_compact<4>, grid, block, 0, s, a);
    case 2: return launch_k(k_kv_compact<2>, grid, block, 0, s, a);
    default: return launch_k(k_kv_compact<1>, grid, block, 0, s, a);
    }
}

}  // namespace ar
