// ar_split.h -- how the attention's line of tiles is cut into the blocks' runs,
// and where a block leaves the parts of items that it shares with others.
// Integer arithmetic only: plain C++ for the host, device code under nvcc.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define AR_SPLIT __device__ __forceinline__
#else
#define AR_SPLIT inline
#endif

namespace ar {

// The run of tiles of block `c` of `blocks`: the first total % blocks blocks take one more.
struct Run {
    long long total;  // tiles of the line
    long long lo;
    long long n;
};

// a / b of a >= 0, b > 0: a 64-bit division takes five times as long as a 32-bit one, and is hardly ever needed.
AR_SPLIT long long divide(long long a, long long b)
{
    return (a | b) <= 0xffffffffll ? static_cast<uint32_t>(a) / static_cast<uint32_t>(b) : a / b;
}

AR_SPLIT Run run_of(long long total, int blocks, int c)
{
    const long long q = divide(total, blocks), r = total - q * blocks;
    return {total, c * q + (c < r ? c : r), q + (c < r)};
}

// The block whose run has tile x.
AR_SPLIT int block_of(long long total, int blocks, long long x)
{
    const long long q = divide(total, blocks), r = total - q * blocks, edge = r * (q + 1);
    return static_cast<int>(x < edge ? divide(x, q + 1) : r + divide(x - edge, q));
}

// The slot of a block's part of an item that others have parts of: a run has one such item at each end at most, and begins
// only the one at its own end.
AR_SPLIT unsigned long long slot_of(int block, bool begins_item) { return 2ull * block + (begins_item ? 1 : 0); }

}  // namespace ar

#undef AR_SPLIT
