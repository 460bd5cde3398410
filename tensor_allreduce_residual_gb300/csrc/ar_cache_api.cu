// ar_cache_api.cu -- the C ABI of the paged key-value cache calls: argument
// checks, launch shapes and dispatch on the element types.  Host code only; it
// allocates nothing.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cmath>
#include <cstdint>

#include "ar.h"
#include "ar_cache.h"

namespace {

constexpr int kMaxHeads = 1024;
constexpr int kMaxHeadDim = 1024;

int esize_of(int dtype) { return dtype == AR_FP32 ? 4 : dtype == AR_FP16 || dtype == AR_BF16 ? 2 : 0; }

int cache_esize_of(int dtype) { return dtype == AR_FP8_E4M3 ? 1 : esize_of(dtype); }

bool aligned(const void* p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

int status_of(cudaError_t e) { return e == cudaSuccess ? AR_OK : AR_ERR_CUDA; }

bool scale_ok(float s) { return std::isfinite(s) && s > 0.0f; }

// The cache with the strides that no element needs (one page, token or head) set to 0, so that they refuse nothing.
ar_kv_cache without_idle_strides(const ar_kv_cache* cache)
{
    ar_kv_cache c{};
    if (cache != nullptr)
        c = *cache;
    c.page_stride = c.pages > 1 ? c.page_stride : 0;
    c.token_stride = c.page_size > 1 ? c.token_stride : 0;
    c.head_stride = c.kv_heads > 1 ? c.head_stride : 0;
    return c;
}

// Sizes, strides and dtype of the cache (all zeros for a NULL one); no pointer is looked at.
int check_sizes(const ar_kv_cache* c)
{
    if (c->pages < 1 || c->page_size < 1 || c->kv_heads < 1 || c->head_dim < 1 || c->batch < 0 ||
        c->max_pages < 1 || c->table_stride < c->max_pages)
        return AR_ERR_INVALID_ARG;
    if (cache_esize_of(c->dtype) == 0 || c->kv_heads > kMaxHeads || c->head_dim > kMaxHeadDim)
        return AR_ERR_UNSUPPORTED;
    const size_t d = static_cast<size_t>(c->head_dim);
    if ((c->pages > 1 && c->page_stride < d) || (c->page_size > 1 && c->token_stride < d) ||
        (c->kv_heads > 1 && c->head_stride < d) || !scale_ok(c->k_scale) || !scale_ok(c->v_scale))
        return AR_ERR_INVALID_ARG;
    return AR_OK;
}

int check_dtypes(int dtype, int cache_dtype)
{
    if (esize_of(dtype) == 0 || !(cache_dtype == dtype || (cache_dtype == AR_FP8_E4M3 && dtype != AR_FP32)))
        return AR_ERR_UNSUPPORTED;
    return AR_OK;
}

bool element_ok(const void* p, size_t esize) { return p != nullptr && aligned(p, esize); }

bool pointers_ok(const ar_kv_cache* c)
{
    const size_t e = static_cast<size_t>(cache_esize_of(c->dtype));
    return element_ok(c->k, e) && element_ok(c->v, e) && element_ok(c->page_table, 4) && element_ok(c->lengths, 4);
}

// Calls f(T{}, CT{}) with the element types of the tensors and of the cache.
template <typename F>
cudaError_t by_dtypes(int dtype, int cache_dtype, F&& f)
{
    const bool small = cache_dtype == AR_FP8_E4M3;
    switch (dtype) {
    case AR_FP32: return f(float{}, float{});
    case AR_FP16: return small ? f(__half{}, __nv_fp8_e4m3{}) : f(__half{}, __half{});
    default: return small ? f(__nv_bfloat16{}, __nv_fp8_e4m3{}) : f(__nv_bfloat16{}, __nv_bfloat16{});
    }
}

uint64_t magic_of(int units) { return ((1ull << 32) + units - 1) / units; }

// Sizes of ar_paged_attention that both it and its workspace size check.
int check_attention(const ar_kv_cache* c, int q_heads)
{
    if (int st = check_sizes(c))
        return st;
    if (q_heads < 1 || q_heads % c->kv_heads != 0)
        return AR_ERR_INVALID_ARG;
    const size_t e = static_cast<size_t>(cache_esize_of(c->dtype));
    if (q_heads > kMaxHeads || c->head_dim > ar::kAttnMaxDim || c->head_dim * e % 16 != 0 ||
        c->page_stride * e % 16 != 0 || c->token_stride * e % 16 != 0 || c->head_stride * e % 16 != 0)
        return AR_ERR_UNSUPPORTED;
    return AR_OK;
}

int group_blocks_of(const ar_kv_cache* c, int q_heads)
{
    const int block_heads = ar::attn_block_heads(cache_esize_of(c->dtype));
    return (q_heads / c->kv_heads + block_heads - 1) / block_heads;
}

// Sequences times key-value heads times blocks of query heads.
size_t attention_items(const ar_kv_cache* c, int q_heads)
{
    return static_cast<size_t>(c->batch) * c->kv_heads * group_blocks_of(c, q_heads);
}

int slot_floats_of(const ar_kv_cache* c, int q_heads)
{
    const int group = q_heads / c->kv_heads, block_heads = ar::attn_block_heads(cache_esize_of(c->dtype));
    return ar::attn_slot_floats(group < block_heads ? group : block_heads, c->head_dim);
}

// Blocks of the attention kernel, at most: no more than there can be tiles.
int attention_blocks(const ar_kv_cache* c, int q_heads)
{
    const long long cap = static_cast<long long>(c->max_pages) * c->page_size;
    const long long tile = ar::attn_tile(cache_esize_of(c->dtype), c->head_dim);
    const long long items = static_cast<long long>(attention_items(c, q_heads));
    const long long tiles = (cap < INT_MAX ? cap : INT_MAX) / tile + 2;
    const long long most = ar::kAttnMaxBlocks;
    return static_cast<int>(items >= most || items * tiles >= most ? most : items * tiles);
}

}  // namespace

extern "C" {

int ar_kv_append(const ar_kv_cache* cache, const ar_append_params* p, ar_stream_t stream)
{
    const ar_kv_cache own = without_idle_strides(cache);
    const ar_kv_cache* const c = &own;
    if (int st = check_sizes(c))
        return st;
    if (p == nullptr)
        return AR_ERR_INVALID_ARG;
    if (int st = check_dtypes(p->dtype, c->dtype))
        return st;
    const bool has_q = p->q != nullptr;
    const size_t d = static_cast<size_t>(c->head_dim);
    if (p->tokens < 0 || (has_q && p->q_heads < 1) || (p->seq_start == nullptr && p->tokens != c->batch) ||
        p->rotary_dim < 0 || p->rotary_dim % 2 != 0 || p->rotary_dim > c->head_dim || !std::isfinite(p->rotary_scale) ||
        (p->rotary_dim > 0 && p->inv_freq == nullptr))
        return AR_ERR_INVALID_ARG;
    if (has_q && p->q_heads > kMaxHeads)
        return AR_ERR_UNSUPPORTED;
    if (p->tokens == 0)
        return AR_OK;
    const size_t e = static_cast<size_t>(esize_of(p->dtype)), ce = static_cast<size_t>(cache_esize_of(c->dtype));
    if (!pointers_ok(c) || !element_ok(p->k, e) || !element_ok(p->v, e) || c->batch < 1 ||
        (has_q && !(element_ok(p->q, e) && element_ok(p->q_out, e))) || !aligned(p->seq_start, 4) ||
        !aligned(p->positions, 4) || !aligned(p->inv_freq, 4))
        return AR_ERR_INVALID_ARG;
    if (p->tokens > 1 && (p->k_stride < d * c->kv_heads || p->v_stride < d * c->kv_heads ||
                          (has_q && (p->q_stride < d * p->q_heads || p->q_out_stride < d * p->q_heads))))
        return AR_ERR_INVALID_ARG;

    ar::AppendArgs a{};
    a.q = p->q;
    a.k = p->k;
    a.v = p->v;
    a.q_out = p->q_out;
    a.k_pages = c->k;
    a.v_pages = c->v;
    a.table = c->page_table;
    a.lengths = c->lengths;
    a.seq_start = p->seq_start;
    a.positions = p->positions;
    a.inv_freq = p->inv_freq;
    a.q_stride = p->tokens > 1 ? p->q_stride : 0;
    a.k_stride = p->tokens > 1 ? p->k_stride : 0;
    a.v_stride = p->tokens > 1 ? p->v_stride : 0;
    a.q_out_stride = p->tokens > 1 ? p->q_out_stride : 0;
    a.page_stride = c->page_stride;
    a.token_stride = c->token_stride;
    a.head_stride = c->head_stride;
    a.capacity = static_cast<uint64_t>(c->max_pages) * static_cast<uint64_t>(c->page_size);
    a.pages = c->pages;
    a.page_size = c->page_size;
    a.table_stride = c->table_stride;
    a.batch = c->batch;
    a.tokens = p->tokens;
    a.q_heads = has_q ? p->q_heads : 0;
    a.kv_heads = c->kv_heads;
    a.head_dim = c->head_dim;
    a.half = p->rotary_dim / 2;
    a.interleaved = p->interleaved != 0;
    a.rotary_scale = p->rotary_scale;
    a.k_scale = c->k_scale;
    a.v_scale = c->v_scale;

    // The vector path: every row and head starts on a vector, the rotated part and its halves are whole vectors.
    const size_t lanes = 16 / e;
    const auto whole = [&](size_t stride) { return stride % lanes == 0; };
    const bool vec = whole(d) && whole(a.interleaved ? 2 * a.half : a.half) && aligned(p->k, 16) && aligned(p->v, 16) &&
                     whole(a.k_stride) && whole(a.v_stride) && aligned(c->k, lanes * ce) && aligned(c->v, lanes * ce) &&
                     whole(c->page_stride) && whole(c->token_stride) && whole(c->head_stride) &&
                     (!has_q || (aligned(p->q, 16) && aligned(p->q_out, 16) && whole(a.q_stride) && whole(a.q_out_stride)));
    const int per = vec ? static_cast<int>(lanes) : 1;
    // A unit of a head whose pairs lie apart is a pair of vectors; the rest of it are single ones.
    a.head_units = c->head_dim / per - (a.interleaved && vec ? 0 : a.half / per);
    a.v_units = c->head_dim / per;
    a.head_magic = magic_of(a.head_units);
    a.v_magic = magic_of(a.v_units);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return status_of(by_dtypes(p->dtype, c->dtype, [&](auto t, auto ct) {
        return ar::launch_append<decltype(t), decltype(ct)>(a, vec, s);
    }));
}

size_t ar_paged_attention_workspace_size(const ar_kv_cache* cache, int q_heads)
{
    const ar_kv_cache own = without_idle_strides(cache);
    const ar_kv_cache* const c = &own;
    if (check_attention(c, q_heads) != AR_OK)
        return 0;
    const size_t blocks = static_cast<size_t>(attention_blocks(c, q_heads));
    const size_t slot = static_cast<size_t>(slot_floats_of(c, q_heads)) * sizeof(float);
    return (attention_items(c, q_heads) * sizeof(int2) + 255) / 256 * 256 + (2 * blocks * slot + 255) / 256 * 256;
}

int ar_paged_attention(const ar_kv_cache* cache, const void* q, size_t q_stride, int q_heads, float scale, int window,
                       float softcap, void* out, float* lse, void* workspace, size_t workspace_bytes, int dtype,
                       ar_stream_t stream)
{
    const ar_kv_cache own = without_idle_strides(cache);
    const ar_kv_cache* const c = &own;
    if (int st = check_attention(c, q_heads))
        return st;
    if (int st = check_dtypes(dtype, c->dtype))
        return st;
    if (!std::isfinite(scale) || window < 0 || !std::isfinite(softcap) || softcap < 0.0f)
        return AR_ERR_INVALID_ARG;
    constexpr float kLog2e = 1.4426950408889634f;
    const float scale2 = scale * c->k_scale * kLog2e * (softcap > 0.0f ? 2.0f / softcap : 1.0f), softcap2 = softcap * kLog2e;
    if (!std::isfinite(scale2) || !std::isfinite(softcap2))
        return AR_ERR_INVALID_ARG;  // an infinite factor would make scores of 0 NaN
    if (c->batch == 0)
        return AR_OK;
    const size_t e = static_cast<size_t>(esize_of(dtype));
    if (!pointers_ok(c) || !element_ok(q, e) || !element_ok(out, e) || !aligned(lse, 4) ||
        (c->batch > 1 && q_stride < static_cast<size_t>(q_heads) * c->head_dim))
        return AR_ERR_INVALID_ARG;
    if (!aligned(q, 16) || !aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(out, 16) ||
        (c->batch > 1 && q_stride * e % 16 != 0) ||
        c->head_dim * e % 16 != 0)
        return AR_ERR_UNSUPPORTED;
    if (workspace == nullptr || !aligned(workspace, 16) ||
        workspace_bytes < ar_paged_attention_workspace_size(c, q_heads))
        return AR_ERR_WORKSPACE;

    const size_t ce = static_cast<size_t>(cache_esize_of(c->dtype));
    const long long cap = static_cast<long long>(c->max_pages) * c->page_size;
    ar::AttnArgs a{};
    a.q = static_cast<const char*>(q);
    a.k = static_cast<const char*>(c->k);
    a.v = static_cast<const char*>(c->v);
    a.out = static_cast<char*>(out);
    a.lse = lse;
    a.blocks_of = static_cast<int2*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + (attention_items(c, q_heads) * sizeof(int2) + 255) / 256 * 256);
    a.table = c->page_table;
    a.lengths = c->lengths;
    a.q_stride = c->batch > 1 ? q_stride * e : 0;
    a.page_stride = c->page_stride * ce;
    a.token_stride = c->token_stride * ce;
    a.head_stride = c->head_stride * ce;
    a.table_stride = c->table_stride;
    a.pages = c->pages;
    a.page_size = c->page_size;
    a.batch = c->batch;
    // m = ceil(2^(31 + l) / d) with 2^l the power of two from d on is below 2^32, and n m >> (31 + l) = n / d below 2^31.
    while ((1ll << a.page_shift) < c->page_size)
        ++a.page_shift;
    a.page_magic = static_cast<uint32_t>(((1ull << (31 + a.page_shift)) + c->page_size - 1) / c->page_size);
    a.capacity = static_cast<int>(cap < INT_MAX - 255 ? cap : INT_MAX - 255);  // a tile's end stays an int
    a.kv_heads = c->kv_heads;
    a.group = q_heads / c->kv_heads;
    a.group_blocks = group_blocks_of(c, q_heads);
    a.block_heads = ar::attn_block_heads(static_cast<int>(ce));
    a.head_dim = c->head_dim;
    a.window = window;
    a.scale2 = scale2;
    a.softcap = softcap;
    a.softcap2 = softcap2;
    a.v_scale = c->v_scale;
    a.fours_magic = magic_of(c->head_dim / 4);
    a.slot_floats = slot_floats_of(c, q_heads);

    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
        return AR_ERR_CUDA;
    const int most = attention_blocks(c, q_heads);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return status_of(by_dtypes(dtype, c->dtype, [&](auto t, auto ct) {
        return ar::launch_attention<decltype(t), decltype(ct)>(a, most, sms, s);
    }));
}

int ar_attention_join(const void* const* partials, const float* const* lse, int R, int rows, int head_dim, void* out,
                      float* lse_out, int dtype, ar_stream_t stream)
{
    if (R < 1 || R > AR_MAX_RANKS || rows < 0 || head_dim < 1)
        return AR_ERR_INVALID_ARG;
    const int esize = esize_of(dtype);
    if (esize == 0)
        return AR_ERR_UNSUPPORTED;
    if (rows == 0)
        return AR_OK;
    if (partials == nullptr || lse == nullptr || !element_ok(out, esize) || !aligned(lse_out, 4))
        return AR_ERR_INVALID_ARG;
    bool packed = aligned(out, 16);
    ar::JoinArgs a{};
    for (int r = 0; r < R; ++r) {
        if (!element_ok(partials[r], esize) || !element_ok(lse[r], 4) || lse[r] == lse_out)
            return AR_ERR_INVALID_ARG;
        packed = packed && aligned(partials[r], 16);
        a.partials[r] = partials[r];
        a.lse[r] = lse[r];
    }
    a.out = out;
    a.lse_out = lse_out;
    a.R = R;
    a.dim = head_dim;
    a.elements = static_cast<uint64_t>(rows) * static_cast<uint64_t>(head_dim);
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    return status_of([&] {
        switch (dtype) {
        case AR_FP32: return ar::launch_join<float>(a, packed, s);
        case AR_FP16: return ar::launch_join<__half>(a, packed, s);
        default: return ar::launch_join<__nv_bfloat16>(a, packed, s);
        }
    }());
}

}  // extern "C"
