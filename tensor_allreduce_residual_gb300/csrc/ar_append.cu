// ar_append.cu -- appending keys and values to a paged cache with the position
// rotation on the way, and the join of R ranks' partial attentions.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>

#include "ar_cache.h"
#include "ar_kernels.cuh"
#include "ar_launch_k.cuh"

namespace ar {

// ---------------------------------------------------------------------------
// Angles.  One turn is 2^64: inv_freq / (2 pi) becomes a 64-bit fraction of a
// turn, whose product with the position wraps around at whole turns by itself,
// so the reduction is exact for any 32-bit position and costs one integer
// multiply (a product in fp32 would be off by 0.06 rad at position 2^20, and
// fp64 runs at 1/64 of the fp32 rate here).  Angles of up to pi a position are
// off by less than 2^-60 rad a position.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint64_t turn_fraction(float inv_freq)
{
    const uint32_t bits = __float_as_uint(inv_freq);
    const int ex = static_cast<int>((bits >> 23) & 255u);
    const uint64_t mant = (bits & 0x7fffffu) | (ex != 0 ? 0x800000u : 0u);
    // inv_freq = mant * 2^(max(ex, 1) - 150); 2^64 / (2 pi) = 0x28be60db9391054a.
    constexpr uint64_t kTurn = 0x28be60db9391054aull;
    const uint64_t lo = mant * kTurn, hi = __umul64hi(mant, kTurn);
    const int shift = 150 - (ex != 0 ? ex : 1);
    uint64_t f;
    if (shift >= 128)
        f = 0;
    else if (shift >= 64)
        f = hi >> (shift - 64);
    else if (shift > 0)
        f = (lo >> shift) | (hi << (64 - shift));
    else
        f = -shift < 64 ? lo << -shift : 0;
    return (bits >> 31) != 0 ? 0 - f : f;
}

__device__ __forceinline__ float2 cos_sin(uint64_t fraction, int position, float scale)
{
    const uint64_t turn = fraction * static_cast<uint64_t>(static_cast<int64_t>(position));
    // The nearest whole quarter, and what is left: at most an eighth of a turn either way, of which fp32 keeps 24 bits however
    // small it is, and so do its sine and cosine, one of which is small near each quarter.
    const uint32_t quarter = static_cast<uint32_t>((turn + (1ull << 61)) >> 62);
    const int64_t rest = static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62));
    float s, c;
    sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);
    const float x = (quarter & 1) != 0 ? s : c, y = (quarter & 1) != 0 ? c : s;
    return make_float2(quarter == 1 || quarter == 2 ? -x * scale : x * scale, quarter >= 2 ? -y * scale : y * scale);
}

// ---------------------------------------------------------------------------
// Units: VEC elements of T (a 16-byte vector, or one element) as fp32.
// ---------------------------------------------------------------------------
template <typename T, bool VEC>
struct Part {
    static constexpr int L = VEC ? Lanes<T>::V : 1;
    __device__ static void load(const void* base, uint64_t e, float* f)
    {
        const T* p = static_cast<const T*>(base) + e;
        if constexpr (VEC)
            Lanes<T>::unpack(*reinterpret_cast<const uint4*>(p), f);
        else
            f[0] = Lanes<T>::to_f(*p);
    }
    __device__ static void store(void* base, uint64_t e, const float* f)
    {
        T* p = static_cast<T*>(base) + e;
        if constexpr (VEC)
            st16(p, Lanes<T>::pack(f));
        else
            *p = Lanes<T>::from_f(f[0]);
    }
};

// Stores a unit of the cache: f / scale, rounded once.
template <typename T, typename CT, bool VEC>
__device__ __forceinline__ void store_cached(void* base, uint64_t e, float* f, float scale)
{
    constexpr int L = Part<T, VEC>::L;
    if (scale != 1.0f) {
#pragma unroll
        for (int l = 0; l < L; ++l)
            f[l] = __fdiv_rn(f[l], scale);
    }
    if constexpr (sizeof(CT) == 1) {
        uint8_t* p = static_cast<uint8_t*>(base) + e;
        if constexpr (VEC) {
            uint32_t w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i], f[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
                const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2], f[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
                w[i] = lo | hi << 16;
            }
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        } else {
            *p = __nv_cvt_float_to_fp8(f[0], __NV_SATFINITE, __NV_E4M3);
        }
    } else {
        Part<T, VEC>::store(base, e, f);
    }
}

__device__ __forceinline__ void rotate(float& x, float& y, float cosine, float sine)
{
    const float u = x, v = y;
    x = u * cosine - v * sine;
    y = v * cosine + u * sine;
}

// Where the table has pair j of a row.  The 2^group_log pairs of a 16-bit vector are read two at a time by threads with the
// vectors beside it: the first two of all vectors, then the next two, so that they lie side by side and meet no bank twice
// (in order, eight bytes a read at steps of 64 met four times and kept the L1 pipe at 79 %: 63.0 against 61.4 us for the
// prompts).  group_log 0: in order, for fp32, whose steps are shorter.
__device__ __forceinline__ int turn_place(int j, int half, int group_log)
{
    const int in = j & ((1 << group_log) - 1);
    return group_log == 0 ? j : ((in >> 1) * (half >> group_log) + (j >> group_log)) * 2 + (j & 1);
}

// ---------------------------------------------------------------------------
// The append.  A block takes up to kAppendMaxTokens rows: it finds their
// sequences (one pass over seq_start, all threads at once: a binary search's
// chain of loads would cost more than the row's copy), fills a table of their
// cosines and sines in shared memory, which all heads of a row share, and then
// walks the rows' units: pairs of vectors that rotate into each other, or
// single vectors.  Bound by HBM for prompts (365 MB in 60 us, 6.1 TB/s; a copy
// of as many bytes takes 55 us) and for single tokens by the chain of loads
// length, page, store (3.0 us for 8 rows).
// What hides the loads is the number of threads: forms that kept several units
// a thread in flight, or a head's cosines and sines in registers, ran fewer of
// them and took 66 to 94 us for the same prompts; hence one unit at a time and
// eight blocks an SM, for whose 32 registers the 16-bit vector kernels spill 24
// to 28 bytes a thread.
// ---------------------------------------------------------------------------
template <typename T, typename CT, bool VEC>
__global__ void __launch_bounds__(kAppendThreads, 8)
k_kv_append(const AppendArgs a)
{
    extern __shared__ __align__(16) float2 s_turn[];  // [rows][half], by turn_place
    __shared__ int s_seq[kAppendMaxTokens];
    __shared__ int s_pos[kAppendMaxTokens];
    __shared__ int64_t s_dst[kAppendMaxTokens];  // element offset in the cache, -1: not cached
    pdl_enter();
    constexpr int L = Part<T, VEC>::L;
    const int t0 = static_cast<int>(blockIdx.x) * a.block_tokens;
    const int rows = min(a.block_tokens, a.tokens - t0);
    const int tid = static_cast<int>(threadIdx.x);

    int first = t0;  // sequence of row t0
    if (a.seq_start != nullptr) {
        first = 0;
        for (int base = 0; base < a.batch; base += kAppendThreads)
            first += __syncthreads_count(base + tid < a.batch && a.seq_start[base + tid + 1] <= t0);
    }
    if (tid < rows) {
        const int t = t0 + tid;
        int b = t, i = 0, n = 1;
        if (a.seq_start != nullptr) {
            b = first;
            while (b < a.batch && a.seq_start[b + 1] <= t)
                ++b;
            if (b < a.batch) {
                const int s = a.seq_start[b];
                i = t - s;
                n = a.seq_start[b + 1] - s;
                if (i < 0)
                    b = a.batch;  // before the first sequence
            }
        }
        int64_t dst = -1, p = 0;
        if (b < a.batch) {
            p = static_cast<int64_t>(a.lengths[b]) - n + i;
            if (p >= 0 && static_cast<uint64_t>(p) < a.capacity) {
                const uint32_t column = static_cast<uint32_t>(p) / static_cast<uint32_t>(a.page_size);  // p is below 2^31
                const int page = a.table[static_cast<uint64_t>(b) * a.table_stride + column];
                if (page >= 0 && page < a.pages)
                    dst = static_cast<int64_t>(static_cast<uint64_t>(page) * a.page_stride +
                                               (static_cast<uint32_t>(p) - column * a.page_size) * a.token_stride);
            }
        }
        s_seq[tid] = b < a.batch ? b : -1;
        s_pos[tid] = a.positions != nullptr ? a.positions[t] : static_cast<int>(p);
        s_dst[tid] = dst;
    }
    __syncthreads();
    // At most two rows in fp32, whose registers are the fewest: the division costs it more than further rows give (2296 rows
    // of 18 heads of 80: 8.1 against 7.0 us).
    const auto row_of = [&](int x, int each, uint64_t magic) {
        if constexpr (sizeof(T) == 4)
            return static_cast<int>(x >= each);
        else
            return a.block_tokens == 1 ? 0 : static_cast<int>(static_cast<uint32_t>(x) * magic >> 32);
    };
    const int group_log = VEC && L == 8 ? (a.interleaved ? 2 : 3) : 0;
    for (int x = tid; x < rows * a.half; x += kAppendThreads) {
        const int row = row_of(x, a.half, a.turn_magic), j = x - row * a.half;
        s_turn[row * a.half + turn_place(j, a.half, group_log)] = cos_sin(turn_fraction(a.inv_freq[j]), s_pos[row], a.rotary_scale);
    }
    __syncthreads();

    const int vectors = a.half >> group_log;
    const int q_units = a.q_heads * a.head_units;
    const int k_units = q_units + a.kv_heads * a.head_units;
    const int all = k_units + a.kv_heads * a.v_units;
    const int pairs = a.half / L;  // units that are pairs (the vector path of interleaved pairs has none)
    for (int x = tid; x < rows * all; x += kAppendThreads) {
        const int row = row_of(x, all, a.row_magic);
        const int u = x - row * all;
        const int64_t dst = s_dst[row];
        const uint64_t t = static_cast<uint64_t>(t0 + row);
        if (s_seq[row] < 0)
            continue;
        float f[L], g[L];
        if (u >= k_units) {
            if (dst < 0)
                continue;
            const uint32_t w = static_cast<uint32_t>(u - k_units);
            const uint32_t head = static_cast<uint32_t>(w * a.v_magic >> 32);
            const uint32_t d = (w - head * a.v_units) * L;
            Part<T, VEC>::load(a.v, t * a.v_stride + head * a.head_dim + d, f);
            store_cached<T, CT, VEC>(a.v_pages, dst + head * a.head_stride + d, f, a.v_scale);
            continue;
        }
        const bool is_q = u < q_units;
        if (!is_q && dst < 0)
            continue;
        const uint32_t w = static_cast<uint32_t>(is_q ? u : u - q_units);
        const uint32_t head = static_cast<uint32_t>(w * a.head_magic >> 32);
        const int c = static_cast<int>(w - head * a.head_units);
        const void* src = is_q ? a.q : a.k;
        const uint64_t from = t * (is_q ? a.q_stride : a.k_stride) + head * a.head_dim;
        const uint64_t to = is_q ? t * a.q_out_stride + head * a.head_dim : dst + head * a.head_stride;
        const float2* turn = s_turn + row * a.half;
        const auto store = [&](int d, float* v) {
            if (is_q)
                Part<T, VEC>::store(a.q_out, to + d, v);
            else
                store_cached<T, CT, VEC>(a.k_pages, to + d, v, a.k_scale);
        };
        if (VEC && a.interleaved) {
            const int d = c * L;
            Part<T, VEC>::load(src, from + d, f);
            if (d < 2 * a.half) {
#pragma unroll
                for (int l = 0; l + 3 < L; l += 4) {
                    const float4 cs = *reinterpret_cast<const float4*>(turn + (L == 8 ? (l / 4 * vectors + c) * 2 : (c * L + l) / 2));
                    rotate(f[l], f[l + 1], cs.x, cs.y);
                    rotate(f[l + 2], f[l + 3], cs.z, cs.w);
                }
            }
            store(d, f);
        } else if (c < pairs) {
            const int d0 = a.interleaved ? 2 * c : c * L;
            const int d1 = a.interleaved ? d0 + 1 : d0 + a.half;
            Part<T, VEC>::load(src, from + d0, f);
            Part<T, VEC>::load(src, from + d1, g);
            if constexpr (VEC) {
#pragma unroll
                for (int l = 0; l < L; l += 2) {
                    const float4 cs = *reinterpret_cast<const float4*>(turn + (L == 8 ? (l / 2 * vectors + c) * 2 : c * L + l));
                    rotate(f[l], g[l], cs.x, cs.y);
                    rotate(f[l + 1], g[l + 1], cs.z, cs.w);
                }
            } else {
                rotate(f[0], g[0], turn[c].x, turn[c].y);
            }
            store(d0, f);
            store(d1, g);
        } else {
            const int d = 2 * a.half + (c - pairs) * L;
            Part<T, VEC>::load(src, from + d, f);
            store(d, f);
        }
    }
}

// Bytes of rows that a block takes, at most, where it takes more than one, and how many blocks run at once.
constexpr int kAppendBytes = 32 * 1024;
constexpr int kAppendBlocks = 152 * 8;

template <typename T, typename CT>
cudaError_t launch_append(const AppendArgs& args, bool vec, cudaStream_t s)
{
    AppendArgs a = args;
    // Few rows: one a block, for latency.  From 1025 on two at least, where that leaves a block under 32 KB: at 8 query heads
    // and one key-value head of 128 bf16 elements 4.3 us either way for 1025 rows, 5.6 against 6.7 for 1500, 10.2 against
    // 13.8 for 4096.  More from 7296 on, as many as leave two blocks for every one that can run: 8192 rows 15.0 us with
    // three, 16.2 with two, 21.7 with one, 32768 rows 41.3 with eight, 44.7 with four, 70.6 with one.  At 24 and 4 heads 8192
    // rows take 26.9 us with two to four and 30.8 with one; at 64 and 8, one row of which is 20 KB, 55.7 with one.
    const int row_units = (a.q_heads + a.kv_heads) * a.head_units + a.kv_heads * a.v_units;
    const int row_bytes = (a.q_heads + 2 * a.kv_heads) * a.head_dim * static_cast<int>(sizeof(T));
    const int by_blocks = a.tokens <= 1024 ? 1 : std::max(2, a.tokens / (2 * kAppendBlocks));
    a.block_tokens = std::max(1, std::min({kAppendBytes / row_bytes, by_blocks, sizeof(T) == 4 ? 2 : kAppendMaxTokens}));
    if (a.block_tokens > 1) {
        a.turn_magic = a.half > 0 ? ((1ull << 32) + a.half - 1) / a.half : 0;
        a.row_magic = ((1ull << 32) + row_units - 1) / row_units;
    }
    const unsigned grid = static_cast<unsigned>((a.tokens + a.block_tokens - 1) / a.block_tokens);
    const size_t smem = static_cast<size_t>(a.block_tokens) * a.half * sizeof(float2);
    return vec ? launch_k(k_kv_append<T, CT, true>, dim3(grid), dim3(kAppendThreads), smem, s, a)
               : launch_k(k_kv_append<T, CT, false>, dim3(grid), dim3(kAppendThreads), smem, s, a);
}

template cudaError_t launch_append<float, float>(const AppendArgs&, bool, cudaStream_t);
template cudaError_t launch_append<__half, __half>(const AppendArgs&, bool, cudaStream_t);
template cudaError_t launch_append<__half, __nv_fp8_e4m3>(const AppendArgs&, bool, cudaStream_t);
template cudaError_t launch_append<__nv_bfloat16, __nv_bfloat16>(const AppendArgs&, bool, cudaStream_t);
template cudaError_t launch_append<__nv_bfloat16, __nv_fp8_e4m3>(const AppendArgs&, bool, cudaStream_t);

// ---------------------------------------------------------------------------
// The join of R partial attentions: a weighted R-way sum, bound by HBM like
// k_sum.  A thread takes 16 bytes of every partial, all loads at once; while
// they come, the block's first threads form the weights of the rows it covers,
// a row a thread, in shared memory.  (Weights formed by every thread for itself
// cost R exponentials each 16 bytes: 12 ranks of 20000 rows of 100 bf16 took
// 20.4 us, 13.7 so.)  Rows that are no whole vectors are taken as one dense
// array all the same: a vector then lies in two rows.
// ---------------------------------------------------------------------------
enum JoinUnits { kJoinElements, kJoinRows, kJoinAcross };  // single elements, vectors of one row, vectors of two rows

// A streaming 16-byte load of what the launch may overwrite: out may be one of the partials, and the read-only path asks for
// memory that nothing writes meanwhile.
__device__ __forceinline__ uint4 ld_stream16_rw(const void* p)
{
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p)
                 : "memory");
    return r;
}

// Rows that a block's elements can touch.
__host__ __device__ inline int join_rows(int lanes, int dim) { return (kFlatThreads * lanes - 1) / dim + 2; }

template <typename T, int UNITS, int R>
__global__ void __launch_bounds__(kFlatThreads)
k_attention_join(const JoinArgs a)
{
    extern __shared__ float s_weights[];  // [rows][R]: a rank's share of the row, -1 where it counts nothing
    pdl_enter();
    using U = Unit<T, UNITS != kJoinElements>;
    constexpr int L = U::L;
    const uint64_t e0 = static_cast<uint64_t>(blockIdx.x) * kFlatThreads * L, e1 = min(e0 + kFlatThreads * L, a.elements);
    const uint64_t i = static_cast<uint64_t>(blockIdx.x) * kFlatThreads + threadIdx.x, e = i * L;
    typename U::raw v[R];
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (i < a.units) {
            if constexpr (UNITS == kJoinElements)
                v[r] = U::load(a.partials[r], i);
            else
                v[r] = ld_stream16_rw(static_cast<const uint4*>(a.partials[r]) + i);
        }
    // A 64-bit division would cost more than the loads of a small row.
    const uint32_t dim = static_cast<uint32_t>(a.dim);
    const auto row_of = [&](uint64_t x) { return a.elements >> 32 == 0 ? static_cast<uint32_t>(x) / dim : x / dim; };
    const uint64_t row0 = row_of(e0);
    for (uint64_t row = row0 + threadIdx.x; row * dim < e1; row += kFlatThreads) {
        float w[R], top = -INFINITY, total = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r)
            w[r] = a.lse[r][row];
#pragma unroll
        for (int r = 0; r < R; ++r)
            top = fmaxf(top, w[r]);
        const float base = top == -INFINITY ? 0.0f : top;
        uint32_t out = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            out |= w[r] == -INFINITY ? 1u << r : 0u;
            w[r] = expf(w[r] - base);
            total += w[r];
        }
        const float inv = 1.0f / total;
#pragma unroll
        for (int r = 0; r < R; ++r)
            s_weights[(row - row0) * R + r] = (out >> r & 1) != 0 ? -1.0f : w[r] * inv;
        if (a.lse_out != nullptr && row * dim >= e0)
            a.lse_out[row] = base + logf(total);
    }
    __syncthreads();
    if (i < a.units) {
        const uint32_t at = static_cast<uint32_t>(e - row0 * dim), local = at / dim;
        // Lanes from `split` on lie in the next row.
        const int split = UNITS == kJoinAcross ? min(static_cast<int>((local + 1) * dim - at), L) : L;
        const float* here = s_weights + local * R;
        float acc[L];
#pragma unroll
        for (int l = 0; l < L; ++l)
            acc[l] = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float w0 = here[r], w1 = UNITS == kJoinAcross && split < L ? here[R + r] : w0;
            float f[L];
            U::to_float(v[r], f);
#pragma unroll
            for (int l = 0; l < L; ++l) {
                const float w = UNITS == kJoinAcross && l >= split ? w1 : w0;
                if (!(w < 0.0f))
                    acc[l] = fmaf(w, f[l], acc[l]);
            }
        }
        U::store(a.out, i, acc);
    } else if (UNITS == kJoinAcross && i == a.units) {  // elements after the last whole vector
        for (uint64_t x = e; x < a.elements; ++x) {
            const float* here = s_weights + static_cast<uint32_t>(x - row0 * dim) / dim * R;
            float acc = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (!(here[r] < 0.0f))
                    acc = fmaf(here[r], Lanes<T>::to_f(static_cast<const T*>(a.partials[r])[x]), acc);
            static_cast<T*>(a.out)[x] = Lanes<T>::from_f(acc);
        }
    }
}

// One kernel for each number of ranks: with a runtime count, and registers for 16, five ranks of 30000 rows of 128 fp32 took
// 25.5 us, 16.0 so.
template <typename T, int UNITS, int R>
static cudaError_t run_join(const JoinArgs& a, dim3 grid, cudaStream_t s)
{
    if constexpr (R < kMaxRanks) {
        if (a.R > R)
            return run_join<T, UNITS, R + 1>(a, grid, s);
    }
    constexpr int L = UNITS == kJoinElements ? 1 : Lanes<T>::V;
    const size_t smem = static_cast<size_t>(join_rows(L, a.dim)) * R * sizeof(float);
    return launch_k(k_attention_join<T, UNITS, R>, grid, dim3(kFlatThreads), smem, s, a);
}

template <typename T>
cudaError_t launch_join(const JoinArgs& args, bool aligned, cudaStream_t s)
{
    constexpr int L = Lanes<T>::V;
    JoinArgs a = args;
    const bool packed = aligned && a.dim >= L, rows = packed && a.dim % L == 0;
    a.units = packed ? a.elements / L : a.elements;
    const uint64_t blocks = (a.units + (packed && !rows) + kFlatThreads - 1) / kFlatThreads;
    if (blocks > static_cast<uint64_t>(INT_MAX))
        return cudaErrorInvalidConfiguration;
    const dim3 grid(static_cast<unsigned>(blocks));
    return rows ? run_join<T, kJoinRows, 1>(a, grid, s)
           : packed ? run_join<T, kJoinAcross, 1>(a, grid, s)
                    : run_join<T, kJoinElements, 1>(a, grid, s);
}

template cudaError_t launch_join<float>(const JoinArgs&, bool, cudaStream_t);
template cudaError_t launch_join<__half>(const JoinArgs&, bool, cudaStream_t);
template cudaError_t launch_join<__nv_bfloat16>(const JoinArgs&, bool, cudaStream_t);

}  // namespace ar
