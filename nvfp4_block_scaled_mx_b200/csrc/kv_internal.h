// kv_internal.h -- launch interfaces of the 4-bit key/value cache kernels (arguments already validated).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mxq {

struct KvAppendArgs {
    const __nv_bfloat16 *k, *v;
    int64_t token_stride[2], head_stride[2];  // elements; [0] of k, [1] of v
    const int32_t* slots;
    const float *g_k, *g_v;
    uint8_t* cache;
    int64_t page_bytes;  // bytes of one head's page
    uint32_t tokens, heads, page_size;
    int num_slots;
    int* status;
};

struct KvReadArgs {
    const uint8_t* cache;
    const int32_t* slots;
    const float *g_k, *g_v;
    __nv_bfloat16 *k_out, *v_out;  // [tokens][heads][D]
    int64_t page_bytes;
    uint32_t tokens, heads, page_size;
    int num_slots;
    int* status;
};

struct KvAttnArgs {
    const __nv_bfloat16* q;
    int64_t q_token_stride, q_head_stride;  // elements
    const uint8_t* cache;
    int64_t page_bytes;  // bytes of one head's page
    const int32_t *table, *lens, *q_start;  // q_start may be null: max_q rows a sequence
    int64_t table_stride;
    const float *g_k, *g_v;
    void* out;   // [T][heads][D]
    float* lse;  // [T][heads] or null
    float* partial;
    int batch, rows_total, max_q, heads, kv_heads, group;
    int page_units;              // units of a page
    uint32_t page_magic;         // unit / page_units = high half of unit * page_magic, for units below 2^26
    int num_pages, max_len;      // max_len = table columns * page_size
    int causal, window, out_f32;
    float scale, inv_grid;
    int* status;
};

int launch_kv_append(int fmt, int rule, int D, const KvAppendArgs& a, cudaStream_t st);
int launch_kv_read(int fmt, int D, const KvReadArgs& a, cudaStream_t st);
int launch_kv_attention(int fmt, int D, KvAttnArgs& a, cudaStream_t st);
// Sequences of more than eight rows on tcgen05 (head size 64 or 128), and the rows of its row tiles.
int launch_kv_attention_rows(int fmt, int D, KvAttnArgs& a, cudaStream_t st);
int kv_rows_tile(int64_t rows);
size_t kv_attention_workspace(int64_t batch, int64_t max_q, int heads, int kv_heads, int D);

// Page bookkeeping.
struct KvPagesArgs {
    const int32_t* seqs;   // [n] rows of the table
    const int32_t* other;  // [n] tokens to add / new lengths / children
    int32_t* table;
    int64_t table_stride;
    int32_t *lens, *refs, *slots, *info;
    int32_t* pairs;  // copy list: [0] count, then source and destination page of each copy
    int n, max_seqs, max_pages, num_pages, page_size, slots_cap;
};

int launch_kv_reserve(const KvPagesArgs& a, uint8_t* cache, int64_t layers, int64_t layer_stride, int64_t page_bytes,
                      cudaStream_t st);
int launch_kv_fork(const KvPagesArgs& a, cudaStream_t st);
int launch_kv_truncate(const KvPagesArgs& a, cudaStream_t st);
int launch_kv_compact(const KvPagesArgs& a, uint8_t* cache, int64_t layers, int64_t layer_stride, int64_t page_bytes,
                      cudaStream_t st);

}  // namespace mxq
