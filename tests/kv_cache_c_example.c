/*
 * kv_cache_c_example.c -- the paged key-value cache calls used from plain C
 * through include/ar.h: two sequences' prompts appended to fp32 pages with the
 * rotation, one-token attention over each half of their tokens, and the join
 * of the halves, on a stream.
 *
 * Usage: kv_cache_c_example <in.bin> <out.bin>
 *   in.bin   fp32 q [2, HEADS, DIM], then k and v [TOKENS, KV_HEADS, DIM]
 *            (the rows of both sequences, LEN0 and LEN1 of them), then
 *            inv_freq [DIM / 2]
 *   out.bin  fp32 out [2, HEADS, DIM] over all tokens, then the join of the
 *            attentions over tokens in even and in odd pages
 * Exit status 0 on success; a failing call prints its status text.
 */
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <cuda_runtime.h>

#include "ar.h"

enum { HEADS = 4, KV_HEADS = 2, DIM = 64, LEN0 = 37, LEN1 = 5, TOKENS = LEN0 + LEN1, PAGE = 8, MAX_PAGES = 5, PAGES = 16 };

static void* device(const void* host, size_t bytes)
{
    void* p = NULL;
    if (cudaMalloc(&p, bytes) != cudaSuccess || cudaMemset(p, 0, bytes) != cudaSuccess ||
        (host != NULL && cudaMemcpy(p, host, bytes, cudaMemcpyHostToDevice) != cudaSuccess)) {
        fprintf(stderr, "device memory: %s\n", cudaGetErrorString(cudaGetLastError()));
        exit(1);
    }
    return p;
}

static void ok(int status, const char* what)
{
    if (status != AR_OK) {
        fprintf(stderr, "%s: %s\n", what, ar_strerror(status));
        exit(1);
    }
}

static int run(int argc, char** argv)
{
    const size_t nq = 2 * HEADS * DIM, nkv = (size_t)TOKENS * KV_HEADS * DIM, in_count = nq + 2 * nkv + DIM / 2;
    float* in = (float*)malloc(in_count * sizeof(float));
    float* out = (float*)malloc(2 * nq * sizeof(float));
    FILE* f = argc == 3 ? fopen(argv[1], "rb") : NULL;
    if (!f || fread(in, sizeof(float), in_count, f) != in_count) {
        fprintf(stderr, "usage: %s in.bin out.bin\n", argv[0]);
        return 2;
    }
    fclose(f);
    float* data = (float*)device(in, in_count * sizeof(float));
    const int table[2][MAX_PAGES] = {{3, 15, 0, 7, 9}, {4, -1, -1, -1, -1}}, lengths[2] = {LEN0, LEN1}, start[3] = {0, LEN0, TOKENS};
    int half_table[2][2][MAX_PAGES];
    for (int h = 0; h < 2; ++h)
        for (int b = 0; b < 2; ++b)
            for (int c = 0; c < MAX_PAGES; ++c)
                half_table[h][b][c] = c % 2 == h ? table[b][c] : -1;
    const size_t pool = (size_t)PAGES * PAGE * KV_HEADS * DIM;

    ar_kv_cache cache;
    memset(&cache, 0, sizeof(cache));
    cache.k = device(NULL, pool * sizeof(float));
    cache.v = device(NULL, pool * sizeof(float));
    cache.dtype = AR_FP32;
    cache.pages = PAGES;
    cache.page_size = PAGE;
    cache.kv_heads = KV_HEADS;
    cache.head_dim = DIM;
    cache.page_stride = (size_t)PAGE * KV_HEADS * DIM;
    cache.token_stride = (size_t)KV_HEADS * DIM;
    cache.head_stride = DIM;
    cache.k_scale = cache.v_scale = 1.0f;
    cache.page_table = (const int*)device(table, sizeof(table));
    cache.batch = 2;
    cache.max_pages = cache.table_stride = MAX_PAGES;
    cache.lengths = (const int*)device(lengths, sizeof(lengths));

    ar_append_params rows;
    memset(&rows, 0, sizeof(rows));
    rows.k = data + nq;
    rows.v = data + nq + nkv;
    rows.tokens = TOKENS;
    rows.dtype = AR_FP32;
    rows.k_stride = rows.v_stride = (size_t)KV_HEADS * DIM;
    rows.seq_start = (const int*)device(start, sizeof(start));
    rows.inv_freq = data + nq + 2 * nkv;
    rows.rotary_dim = DIM;
    rows.rotary_scale = 1.0f;

    cudaStream_t stream;
    if (cudaStreamCreate(&stream) != cudaSuccess)
        return 1;
    ok(ar_kv_append(&cache, &rows, (ar_stream_t)stream), "ar_kv_append");

    const size_t ws_bytes = ar_paged_attention_workspace_size(&cache, HEADS);
    void* ws = device(NULL, ws_bytes);
    float* results = (float*)device(NULL, 4 * nq * sizeof(float));   /* whole, joined, the halves */
    float* lse = (float*)device(NULL, 2 * 2 * HEADS * sizeof(float));
    ok(ar_paged_attention(&cache, data, (size_t)HEADS * DIM, HEADS, 0.125f, 0, 0.0f, results, NULL, ws, ws_bytes, AR_FP32,
                          (ar_stream_t)stream), "ar_paged_attention");
    const void* parts[2];
    const float* part_lse[2];
    for (int h = 0; h < 2; ++h) {
        ar_kv_cache half = cache;
        half.page_table = (const int*)device(half_table[h], sizeof(half_table[h]));
        parts[h] = results + (2 + h) * nq;
        part_lse[h] = lse + h * 2 * HEADS;
        ok(ar_paged_attention(&half, data, (size_t)HEADS * DIM, HEADS, 0.125f, 0, 0.0f, (void*)parts[h], (float*)part_lse[h], ws,
                              ws_bytes, AR_FP32, (ar_stream_t)stream), "ar_paged_attention over a half");
    }
    ok(ar_attention_join(parts, part_lse, 2, 2 * HEADS, DIM, results + nq, NULL, AR_FP32, (ar_stream_t)stream), "ar_attention_join");
    if (cudaStreamSynchronize(stream) != cudaSuccess ||
        cudaMemcpy(out, results, 2 * nq * sizeof(float), cudaMemcpyDeviceToHost) != cudaSuccess) {
        fprintf(stderr, "results: %s\n", cudaGetErrorString(cudaGetLastError()));
        return 1;
    }
    f = fopen(argv[2], "wb");
    if (!f || fwrite(out, sizeof(float), 2 * nq, f) != 2 * nq)
        return 2;
    fclose(f);
    free(in);
    free(out);
    return 0;
}

int main(int argc, char** argv)
{
    int failed = run(argc, argv);
    if (!failed && cudaDeviceReset() != cudaSuccess)
        failed = 1;
    if (!failed)
        failed = run(argc, argv);
    if (!failed)
        printf("kv_cache_c_example: ok\n");
    return failed;
}
