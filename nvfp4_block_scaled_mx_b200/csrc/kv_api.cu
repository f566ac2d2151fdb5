// kv_api.cu -- the extern "C" entry points of the 4-bit key/value cache: argument checks (before any
// launch) and dispatch.
#include "kv_internal.h"
#include "kv.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int64_t kInt = int64_t(1) << 31;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool fmt_ok(int fmt) { return fmt == MXQ_MXFP4 || fmt == MXQ_NVFP4; }

bool cache_ok(int64_t num_pages, int page_size, int kv_heads, int head_dim) {
    return (head_dim == 64 || head_dim == 128 || head_dim == 256) && kv_heads >= 1 && kv_heads <= 65536 &&
           page_size >= 16 && page_size <= 1024 && page_size % 16 == 0 && num_pages >= 1 && num_pages < kInt &&
           num_pages * page_size < kInt;
}

int64_t head_page_bytes(int page_size, int head_dim, int fmt) {
    return static_cast<int64_t>(page_size / 16) * kv_unit_bytes(head_dim, fmt);
}

// An element stride that keeps 16-byte loads aligned.
bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < (int64_t(1) << 40); }

bool tokens_ok(int64_t tokens, int kv_heads, int head_dim) {
    return tokens >= 0 && tokens < kInt && tokens * 2 * kv_heads * (head_dim / 32) < kInt - 1024;
}

// The parts that all page calls share; rows is the number of table rows a call may name.
int check_pages(int64_t n, const void* table, int64_t rows, int64_t stride, int64_t max_pages, const void* lens,
                const void* refs, int64_t num_pages, int page_size, const void* info) {
    if (!table || !lens || !refs || !info) return MXQ_ERR_NULL;
    if (n < 0 || n > MXQ_KV_MAX_SEQS || rows < 1 || rows > MXQ_KV_MAX_TABLE || max_pages < 1 || stride < max_pages ||
        stride >= kInt || page_size < 16 || page_size > 1024 || page_size % 16 != 0 || num_pages < 1 ||
        num_pages >= kInt || num_pages * page_size >= kInt || max_pages * page_size >= kInt)
        return MXQ_ERR_SHAPE;
    if (!aligned(table, 4) || !aligned(lens, 4) || !aligned(refs, 4) || !aligned(info, 4)) return MXQ_ERR_ALIGN;
    return MXQ_OK;
}

int check_layers(const void* cache, int64_t layers, int64_t layer_stride, int64_t page_bytes, int64_t num_pages) {
    if (!cache) return MXQ_ERR_NULL;
    if (layers < 1 || layers > 65536 || page_bytes < 16 || page_bytes >= kInt || page_bytes % 16 != 0 ||
        layer_stride % 16 != 0 || layer_stride < num_pages * page_bytes || layer_stride >= (int64_t(1) << 44))
        return MXQ_ERR_SHAPE;
    return aligned(cache, 16) ? MXQ_OK : MXQ_ERR_ALIGN;
}

KvPagesArgs pages_args(const int32_t* seqs, const int32_t* other, int64_t n, int32_t* table, int64_t rows, int64_t stride,
                       int64_t max_pages, int32_t* lens, int32_t* refs, int64_t num_pages, int page_size, int32_t* info) {
    KvPagesArgs a = {};
    a.seqs = seqs;
    a.other = other;
    a.table = table;
    a.table_stride = stride;
    a.lens = lens;
    a.refs = refs;
    a.info = info;
    a.n = static_cast<int>(n);
    a.max_seqs = static_cast<int>(rows);
    a.max_pages = static_cast<int>(max_pages);
    a.num_pages = static_cast<int>(num_pages);
    a.page_size = page_size;
    return a;
}

}  // namespace
}  // namespace mxq

using namespace mxq;

extern "C" {

int mxq_kv_unit_bytes(int head_dim, mxq_fmt fmt, size_t* bytes) {
    if (!fmt_ok(fmt)) return MXQ_ERR_UNSUPPORTED;
    if (!bytes) return MXQ_ERR_NULL;
    if (head_dim != 64 && head_dim != 128 && head_dim != 256) return MXQ_ERR_SHAPE;
    *bytes = static_cast<size_t>(kv_unit_bytes(head_dim, fmt));
    return MXQ_OK;
}

int mxq_kv_append(const void* k, const void* v, int64_t tokens, int kv_heads, int head_dim, int64_t k_token_stride,
                  int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const int32_t* slots,
                  mxq_fmt fmt, mxq_rule rule, const float* g_k, const float* g_v, void* cache, int64_t num_pages,
                  int page_size, mxq_stream_t stream) {
    if (!fmt_ok(fmt) || (fmt == MXQ_MXFP4 && rule != MXQ_RULE_EVEN && rule != MXQ_RULE_CEIL)) return MXQ_ERR_UNSUPPORTED;
    if (!cache || (tokens != 0 && (!k || !v || !slots)) || (fmt == MXQ_NVFP4 && (!g_k || !g_v))) return MXQ_ERR_NULL;
    if (!cache_ok(num_pages, page_size, kv_heads, head_dim) || !tokens_ok(tokens, kv_heads, head_dim) ||
        !stride_ok(k_token_stride) || !stride_ok(k_head_stride) || !stride_ok(v_token_stride) || !stride_ok(v_head_stride))
        return MXQ_ERR_SHAPE;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(cache, 16) || !aligned(slots, 4) || !aligned(g_k, 4) ||
        !aligned(g_v, 4))
        return MXQ_ERR_ALIGN;
    int rc = check_device();
    if (rc != MXQ_OK) return rc;
    if (tokens == 0) return MXQ_OK;
    KvAppendArgs a = {};
    a.k = static_cast<const __nv_bfloat16*>(k);
    a.v = static_cast<const __nv_bfloat16*>(v);
    a.token_stride[0] = k_token_stride;
    a.token_stride[1] = v_token_stride;
    a.head_stride[0] = k_head_stride;
    a.head_stride[1] = v_head_stride;
    a.slots = slots;
    a.g_k = g_k;
    a.g_v = g_v;
    a.cache = static_cast<uint8_t*>(cache);
    a.page_bytes = head_page_bytes(page_size, head_dim, fmt);
    a.tokens = static_cast<uint32_t>(tokens);
    a.heads = static_cast<uint32_t>(kv_heads);
    a.page_size = static_cast<uint32_t>(page_size);
    a.num_slots = static_cast<int>(num_pages * page_size);
    a.status = status_ptr();
    return launch_kv_append(fmt, rule, head_dim, a, reinterpret_cast<cudaStream_t>(stream));
}

int mxq_kv_read(const void* cache, int64_t num_pages, int page_size, int kv_heads, int head_dim, mxq_fmt fmt,
                const int32_t* slots, int64_t tokens, const float* g_k, const float* g_v, void* k_out, void* v_out,
                mxq_stream_t stream) {
    if (!fmt_ok(fmt)) return MXQ_ERR_UNSUPPORTED;
    if (!cache || (tokens != 0 && (!slots || !k_out || !v_out)) || (fmt == MXQ_NVFP4 && (!g_k || !g_v)))
        return MXQ_ERR_NULL;
    if (!cache_ok(num_pages, page_size, kv_heads, head_dim) || !tokens_ok(tokens, kv_heads, head_dim)) return MXQ_ERR_SHAPE;
    if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(cache, 16) || !aligned(slots, 4) || !aligned(g_k, 4) ||
        !aligned(g_v, 4))
        return MXQ_ERR_ALIGN;
    int rc = check_device();
    if (rc != MXQ_OK) return rc;
    if (tokens == 0) return MXQ_OK;
    KvReadArgs a = {};
    a.cache = static_cast<const uint8_t*>(cache);
    a.slots = slots;
    a.g_k = g_k;
    a.g_v = g_v;
    a.k_out = static_cast<__nv_bfloat16*>(k_out);
    a.v_out = static_cast<__nv_bfloat16*>(v_out);
    a.page_bytes = head_page_bytes(page_size, head_dim, fmt);
    a.tokens = static_cast<uint32_t>(tokens);
    a.heads = static_cast<uint32_t>(kv_heads);
    a.page_size = static_cast<uint32_t>(page_size);
    a.num_slots = static_cast<int>(num_pages * page_size);
    a.status = status_ptr();
    return launch_kv_read(fmt, head_dim, a, reinterpret_cast<cudaStream_t>(stream));
}

size_t mxq_kv_attention_workspace_size(int64_t batch, int64_t max_q, int heads, int kv_heads, int head_dim) {
    if (batch < 0 || batch >= kInt || max_q < 1 || kv_heads < 1 || heads < 1 || heads % kv_heads != 0 ||
        max_q >= kInt || max_q * (heads / kv_heads) >= (int64_t(1) << 28) ||
        (head_dim != 64 && head_dim != 128 && head_dim != 256))
        return 0;
    return kv_attention_workspace(batch, max_q, heads, kv_heads, head_dim);
}

int mxq_kv_attention(const void* q, int64_t rows, int64_t q_token_stride, int64_t q_head_stride, const void* cache,
                     int64_t num_pages, int page_size, int heads, int kv_heads, int head_dim, mxq_fmt fmt,
                     const int32_t* block_table, int64_t table_stride, int64_t max_pages, const int32_t* kv_lens,
                     int64_t batch, const int32_t* q_start, int64_t max_q, float scale, int causal, int64_t window,
                     const float* g_k, const float* g_v, mxq_out out_type, void* out, float* lse, void* workspace,
                     size_t ws_bytes, mxq_stream_t stream) {
    if (!fmt_ok(fmt) || (out_type != MXQ_OUT_BF16 && out_type != MXQ_OUT_FP32)) return MXQ_ERR_UNSUPPORTED;
    const bool none = rows == 0 || batch == 0;
    if (!cache || (!none && (!q || !block_table || !kv_lens || !out || !workspace)) ||
        (fmt == MXQ_NVFP4 && (!g_k || !g_v)))
        return MXQ_ERR_NULL;
    if (!cache_ok(num_pages, page_size, kv_heads, head_dim) || heads < 1 || heads > (1 << 20) || heads % kv_heads != 0 ||
        batch < 0 || batch >= (int64_t(1) << 24) || rows < 0 || rows >= kInt || max_q < 1 || max_q >= kInt ||
        max_q * (heads / kv_heads) >= (int64_t(1) << 28) || max_pages < 1 || table_stride < max_pages ||
        table_stride >= (int64_t(1) << 40) || max_pages * page_size > (int64_t(1) << 30) - 1024 || window < 0 || window >= kInt ||
        !stride_ok(q_token_stride) || !stride_ok(q_head_stride) || (!q_start && rows != batch * max_q))
        return MXQ_ERR_SHAPE;
    if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(workspace, 16) || !aligned(block_table, 4) ||
        !aligned(kv_lens, 4) || !aligned(q_start, 4) || !aligned(lse, 4) || !aligned(g_k, 4) || !aligned(g_v, 4))
        return MXQ_ERR_ALIGN;
    int rc = check_device();
    if (rc != MXQ_OK) return rc;
    if (none) return MXQ_OK;
    if (ws_bytes < kv_attention_workspace(batch, max_q, heads, kv_heads, head_dim)) return MXQ_ERR_WORKSPACE;
    KvAttnArgs a = {};
    a.q = static_cast<const __nv_bfloat16*>(q);
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.cache = static_cast<const uint8_t*>(cache);
    a.page_bytes = head_page_bytes(page_size, head_dim, fmt);
    a.table = block_table;
    a.table_stride = table_stride;
    a.lens = kv_lens;
    a.q_start = q_start;
    a.g_k = g_k;
    a.g_v = g_v;
    a.out = out;
    a.lse = lse;
    a.partial = static_cast<float*>(workspace);
    a.batch = static_cast<int>(batch);
    a.rows_total = static_cast<int>(rows);
    a.max_q = static_cast<int>(max_q);
    a.heads = heads;
    a.kv_heads = kv_heads;
    a.group = heads / kv_heads;
    a.page_units = page_size / 16;
    a.page_magic = a.page_units == 1 ? 0 : static_cast<uint32_t>(((uint64_t(1) << 32) + a.page_units - 1) / a.page_units);
    a.num_pages = static_cast<int>(num_pages);
    a.max_len = static_cast<int>(max_pages * page_size);
    a.causal = causal != 0;
    // No sequence is longer than 2^30, so a wider window is no other; a row's own place may be negative, down to
    // -2^28 (fewer cached tokens than query rows), and the kernels subtract the window from it in 32 bits.
    a.window = static_cast<int>(window < (int64_t(1) << 30) ? window : int64_t(1) << 30);
    a.out_f32 = out_type == MXQ_OUT_FP32;
    a.scale = scale;
    a.status = status_ptr();
    return launch_kv_attention(fmt, head_dim, a, reinterpret_cast<cudaStream_t>(stream));
}

size_t mxq_kv_reserve_workspace_size(int64_t n) {
    return n < 0 || n > MXQ_KV_MAX_SEQS ? 0 : static_cast<size_t>(16 + 8 * n);
}

int mxq_kv_reserve(const int32_t* seqs, const int32_t* add, int64_t n, int32_t* block_table, int64_t table_rows,
                   int64_t table_stride, int64_t max_pages, int32_t* kv_lens, int32_t* refs, int64_t num_pages,
                   int page_size, void* cache, int64_t layers, int64_t layer_stride, int64_t page_bytes, int32_t* slots,
                   int64_t slots_cap, int32_t* info, void* workspace, size_t ws_bytes, mxq_stream_t stream) {
    int rc = check_pages(n, block_table, table_rows, table_stride, max_pages, kv_lens, refs, num_pages, page_size, info);
    if (rc != MXQ_OK) return rc;
    if ((rc = check_layers(cache, layers, layer_stride, page_bytes, num_pages)) != MXQ_OK) return rc;
    if (n != 0 && (!seqs || !add || !workspace)) return MXQ_ERR_NULL;
    if (slots_cap < 0 || slots_cap >= kInt) return MXQ_ERR_SHAPE;
    if (!aligned(seqs, 4) || !aligned(add, 4) || !aligned(slots, 4) || !aligned(workspace, 16)) return MXQ_ERR_ALIGN;
    if (n != 0 && ws_bytes < mxq_kv_reserve_workspace_size(n)) return MXQ_ERR_WORKSPACE;
    if ((rc = check_device()) != MXQ_OK) return rc;
    KvPagesArgs a = pages_args(seqs, add, n, block_table, table_rows, table_stride, max_pages, kv_lens, refs, num_pages,
                               page_size, info);
    a.slots = slots;
    a.slots_cap = slots ? static_cast<int>(slots_cap) : 0;
    a.pairs = static_cast<int32_t*>(workspace);  // (n = 0 needs none)
    return launch_kv_reserve(a, static_cast<uint8_t*>(cache), layers, layer_stride, page_bytes,
                             reinterpret_cast<cudaStream_t>(stream));
}

int mxq_kv_fork(const int32_t* parents, const int32_t* children, int64_t n, int32_t* block_table, int64_t table_rows,
                int64_t table_stride, int64_t max_pages, int32_t* kv_lens, int32_t* refs, int64_t num_pages,
                int page_size, int32_t* info, mxq_stream_t stream) {
    int rc = check_pages(n, block_table, table_rows, table_stride, max_pages, kv_lens, refs, num_pages, page_size, info);
    if (rc != MXQ_OK) return rc;
    if (n != 0 && (!parents || !children)) return MXQ_ERR_NULL;
    if (!aligned(parents, 4) || !aligned(children, 4)) return MXQ_ERR_ALIGN;
    if ((rc = check_device()) != MXQ_OK) return rc;
    return launch_kv_fork(pages_args(parents, children, n, block_table, table_rows, table_stride, max_pages, kv_lens, refs,
                                     num_pages, page_size, info),
                          reinterpret_cast<cudaStream_t>(stream));
}

int mxq_kv_truncate(const int32_t* seqs, const int32_t* new_lens, int64_t n, int32_t* block_table, int64_t table_rows,
                    int64_t table_stride, int64_t max_pages, int32_t* kv_lens, int32_t* refs, int64_t num_pages,
                    int page_size, int32_t* info, mxq_stream_t stream) {
    int rc = check_pages(n, block_table, table_rows, table_stride, max_pages, kv_lens, refs, num_pages, page_size, info);
    if (rc != MXQ_OK) return rc;
    if (n != 0 && (!seqs || !new_lens)) return MXQ_ERR_NULL;
    if (!aligned(seqs, 4) || !aligned(new_lens, 4)) return MXQ_ERR_ALIGN;
    if ((rc = check_device()) != MXQ_OK) return rc;
    return launch_kv_truncate(pages_args(seqs, new_lens, n, block_table, table_rows, table_stride, max_pages, kv_lens, refs,
                                         num_pages, page_size, info),
                              reinterpret_cast<cudaStream_t>(stream));
}

size_t mxq_kv_compact_workspace_size(int64_t num_pages) {
    return num_pages < 1 || num_pages >= kInt ? 0 : static_cast<size_t>(16 + 12 * num_pages);
}

int mxq_kv_compact(int32_t* block_table, int64_t table_rows, int64_t table_stride, int64_t max_pages,
                   const int32_t* kv_lens, int32_t* refs, int64_t num_pages, int page_size, void* cache, int64_t layers,
                   int64_t layer_stride, int64_t page_bytes, int32_t* info, void* workspace, size_t ws_bytes,
                   mxq_stream_t stream) {
    int rc = check_pages(0, block_table, table_rows, table_stride, max_pages, kv_lens, refs, num_pages, page_size, info);
    if (rc != MXQ_OK) return rc;
    if ((rc = check_layers(cache, layers, layer_stride, page_bytes, num_pages)) != MXQ_OK) return rc;
    if (!workspace) return MXQ_ERR_NULL;
    if (!aligned(workspace, 16)) return MXQ_ERR_ALIGN;
    if (ws_bytes < mxq_kv_compact_workspace_size(num_pages)) return MXQ_ERR_WORKSPACE;
    if ((rc = check_device()) != MXQ_OK) return rc;
    KvPagesArgs a = pages_args(nullptr, nullptr, 0, block_table, table_rows, table_stride, max_pages,
                               const_cast<int32_t*>(kv_lens), refs, num_pages, page_size, info);
    a.pairs = static_cast<int32_t*>(workspace);
    return launch_kv_compact(a, static_cast<uint8_t*>(cache), layers, layer_stride, page_bytes,
                             reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
