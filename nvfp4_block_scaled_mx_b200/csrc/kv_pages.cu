// kv_pages.cu -- bookkeeping of the cache's pages on the device: reference counts, block tables, lengths.
//
// A call checks all of its sequences before it changes anything, and either does all of its work or
// none (info[0] says which).  Table work is small and latency-bound, so it is one launch of a single
// cluster of eight CTAs, whose phases are separated by the cluster's hardware barrier instead of by
// launches.  Every CTA checks the whole call for itself (at most 4096 sequences), so no verdict has to
// be exchanged.  Pages are handed out lowest index first, in the order of the call's sequences: results
// do not depend on timing.  Page contents move in a second kernel that reads the list of copies.
#include <cooperative_groups.h>

#include <atomic>

#include "kv.cuh"
#include "kv_internal.h"
#include "mxq_internal.h"

namespace cg = cooperative_groups;

namespace mxq {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 1024;
constexpr int kAll = kCluster * kThreads;

constexpr int kBadIndex = -1;   // a sequence outside the table, given twice, or in an unfit state
constexpr int kBadLength = -2;  // a count or length that is negative, too long, or more slots than slots[] holds
constexpr int kNoPages = -3;    // fewer free pages than the call needs

struct Shared {
    uint32_t seen[MXQ_KV_MAX_TABLE / 32];  // rows named by the call
    int64_t warp_sums[32];
    int64_t total[2];                      // this CTA's total of each scan over the cluster, read by the others
    int64_t totals[kCluster];
    int verdict;
};

struct Reserve : Shared {
    int need[MXQ_KV_MAX_SEQS + 1];     // pages needed by the sequences in front
    int add[MXQ_KV_MAX_SEQS + 1];      // tokens of the sequences in front
    uint16_t copy[MXQ_KV_MAX_SEQS];    // number of the sequence's tail page among those copied, kNoCopy
};
constexpr uint16_t kNoCopy = 0xFFFFu;

__device__ __forceinline__ int pages_for(int64_t len, int page_size) {
    return static_cast<int>((len + page_size - 1) / page_size);
}

// Exclusive scan over the CTA's threads; `all` receives the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, Shared& sh, int64_t& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sh.warp_sums[warp] = x;
    __syncthreads();
    int64_t before = 0, sum = 0;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        const int64_t y = sh.warp_sums[k];
        before += k < warp ? y : 0;
        sum += y;
    }
    all = sum;
    return before + x - v;
}

// The same over the cluster, CTAs in rank order; `slot` 0 or 1, another for each scan of a kernel.  A cluster
// barrier has to follow before a CTA leaves: others read its total.
__device__ __forceinline__ int64_t cluster_scan(int64_t v, Shared& sh, int slot, int64_t& all) {
    cg::cluster_group cl = cg::this_cluster();
    int64_t mine;
    const int64_t x = block_scan(v, sh, mine);
    if (threadIdx.x == 0) sh.total[slot] = mine;
    cl.sync();
    if (threadIdx.x < kCluster) sh.totals[threadIdx.x] = *cl.map_shared_rank(&sh.total[slot], threadIdx.x);
    __syncthreads();
    int64_t before = 0, sum = 0;
#pragma unroll
    for (unsigned k = 0; k < kCluster; ++k) {
        const int64_t y = sh.totals[k];
        before += k < cl.block_rank() ? y : 0;
        sum += y;
    }
    all = sum;
    return before + x;
}

// Marks row r as named; false if it was already or is outside the table.
__device__ __forceinline__ bool claim(Shared& sh, int r, int rows) {
    if (r < 0 || r >= rows) return false;
    const uint32_t bit = 1u << (r & 31);
    return (atomicOr(&sh.seen[r >> 5], bit) & bit) == 0;
}

__device__ __forceinline__ void clear_seen(Shared& sh, int rows) {
    for (int i = threadIdx.x; i < (rows + 31) / 32; i += kThreads) sh.seen[i] = 0;
    if (threadIdx.x == 0) sh.verdict = 0;
    __syncthreads();
}

// The call's verdict: the most negative code of any thread (every CTA comes to the same one).
__device__ __forceinline__ int agree(Shared& sh, int code) {
    if (code < 0) atomicMin(&sh.verdict, code);
    __syncthreads();
    return sh.verdict;
}

// Sequences are spread over the cluster's threads in groups of `per` threads (a power of two).
__device__ __forceinline__ int group_size(int n) {
    int per = 32;
    while (per < kAll && 2 * per * n <= kAll) per *= 2;
    return per;
}

__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads) kv_fork_kernel(const KvPagesArgs a, int* status) {
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    pdl_launch_dependents();
    pdl_wait();
    clear_seen(sh, a.max_seqs);
    int code = 0;
    int64_t shared = 0;
    for (int i = threadIdx.x; i < a.n; i += kThreads) {
        const int c = a.other[i];
        if (!claim(sh, c, a.max_seqs) || a.lens[c] != 0) code = min(code, kBadIndex);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.n; i += kThreads) {
        const int p = a.seqs[i];
        if (p < 0 || p >= a.max_seqs || (sh.seen[p >> 5] >> (p & 31) & 1u)) {  // a parent that is also a child
            code = min(code, kBadIndex);
        } else if (a.lens[p] < 0 || pages_for(a.lens[p], a.page_size) > a.max_pages) {
            code = min(code, kBadLength);
        } else {
            shared += pages_for(a.lens[p], a.page_size);
        }
    }
    code = agree(sh, code);
    int64_t all;
    block_scan(shared, sh, all);
    const int me = cl.block_rank() * kThreads + threadIdx.x;
    if (me == 0) {
        a.info[0] = code;
        a.info[1] = code < 0 ? 0 : static_cast<int>(all);
    }
    cl.sync();  // every CTA has read what is changed below
    if (code < 0) return;
    const int per = group_size(a.n);
    for (int i = me / per; i < a.n; i += kAll / per) {
        const int p = a.seqs[i], c = a.other[i], len = a.lens[p], pages = pages_for(len, a.page_size);
        for (int k = me % per; k < pages; k += per) {
            const int pg = a.table[p * a.table_stride + k];
            a.table[c * a.table_stride + k] = pg;
            if (pg >= 0 && pg < a.num_pages)
                atomicAdd(&a.refs[pg], 1);
            else
                kv_status(status, kStatusKvPage);
        }
        if (me % per == 0) a.lens[c] = len;
    }
}

__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads)
    kv_truncate_kernel(const KvPagesArgs a, int* status) {
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    pdl_launch_dependents();
    pdl_wait();
    clear_seen(sh, a.max_seqs);
    int code = 0;
    int64_t dropped = 0;
    for (int i = threadIdx.x; i < a.n; i += kThreads) {
        const int s = a.seqs[i], to = a.other[i];
        if (!claim(sh, s, a.max_seqs))
            code = min(code, kBadIndex);
        else if (to < 0 || to > a.lens[s] || pages_for(a.lens[s], a.page_size) > a.max_pages)
            code = min(code, kBadLength);
        else
            dropped += pages_for(a.lens[s], a.page_size) - pages_for(to, a.page_size);
    }
    code = agree(sh, code);
    int64_t all;
    block_scan(dropped, sh, all);
    const int me = cl.block_rank() * kThreads + threadIdx.x;
    if (me == 0) {
        a.info[0] = code;
        a.info[1] = code < 0 ? 0 : static_cast<int>(all);
    }
    if (code < 0) return;  // the same verdict in every CTA: none waits for another
    const int per = group_size(a.n);
    for (int i = me / per; i < a.n; i += kAll / per) {
        const int s = a.seqs[i], to = pages_for(a.other[i], a.page_size), from = pages_for(a.lens[s], a.page_size);
        for (int k = to + me % per; k < from; k += per) {
            int* at = a.table + s * a.table_stride + k;
            const int pg = *at;
            if (pg >= 0 && pg < a.num_pages)
                atomicSub(&a.refs[pg], 1);
            else
                kv_status(status, kStatusKvPage);
            *at = -1;
        }
    }
    cl.sync();  // lengths change once nobody reads them any more
    for (int i = me; i < a.n; i += kAll) a.lens[a.seqs[i]] = a.other[i];
}

// Index i with prefix[i] <= r < prefix[i + 1].
__device__ __forceinline__ int owner(const int* prefix, int n, int r) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= r)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads) kv_reserve_kernel(const KvPagesArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    Reserve& sh = *reinterpret_cast<Reserve*>(smem);
    cg::cluster_group cl = cg::this_cluster();
    pdl_launch_dependents();
    pdl_wait();
    clear_seen(sh, a.max_seqs);
    int code = 0;
    // four consecutive sequences a thread, so that one scan gives the prefixes: of pages (low half) and of
    // copies (from bit 40), and of tokens
    constexpr int PER = MXQ_KV_MAX_SEQS / kThreads;
    int64_t need[PER], add[PER], needs = 0, adds = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
        const int i = threadIdx.x * PER + k;
        need[k] = add[k] = 0;
        if (i >= a.n) continue;
        const int s = a.seqs[i];
        if (!claim(sh, s, a.max_seqs)) {
            code = min(code, kBadIndex);
            continue;
        }
        const int64_t len = a.lens[s], more = a.other[i];
        if (len < 0 || more < 0 || len + more > static_cast<int64_t>(a.max_pages) * a.page_size ||
            len + more > 0x7fffffff) {
            code = min(code, kBadLength);
            continue;
        }
        add[k] = more;
        need[k] = pages_for(len + more, a.page_size) - pages_for(len, a.page_size);
        if (more > 0 && len % a.page_size != 0) {
            const int pg = a.table[s * a.table_stride + len / a.page_size];
            if (pg < 0 || pg >= a.num_pages)
                code = min(code, kBadIndex);
            else if (a.refs[pg] > 1)  // a shared page that is not full is copied before it is written
                need[k] += 1 + (int64_t(1) << 40);
        }
        needs += need[k];
        adds += add[k];
    }
    int64_t want, tokens;
    int64_t n0 = block_scan(needs, sh, want), a0 = block_scan(adds, sh, tokens);
    const int copies = static_cast<int>(want >> 40);
    want &= (int64_t(1) << 40) - 1;
    if (want > a.num_pages) code = min(code, kNoPages);
    if ((a.slots && tokens > a.slots_cap) || tokens > 0x7fffffff) code = min(code, kBadLength);
    code = agree(sh, code);
    if (code == 0) {
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int i = threadIdx.x * PER + k;
            if (i > a.n) break;
            sh.need[i] = static_cast<int>(n0 & ((int64_t(1) << 40) - 1));
            sh.add[i] = static_cast<int>(a0);
            if (i < a.n) sh.copy[i] = need[k] >> 40 ? static_cast<uint16_t>(n0 >> 40) : kNoCopy;
            n0 += need[k];
            a0 += add[k];
        }
        if (threadIdx.x == kThreads - 1 && a.n == MXQ_KV_MAX_SEQS) {
            sh.need[a.n] = static_cast<int>(want);
            sh.add[a.n] = static_cast<int>(tokens);
        }
    }
    // free pages in this thread's stretch of the reference counts
    const int me = cl.block_rank() * kThreads + threadIdx.x;
    const int each = (a.num_pages + kAll - 1) / kAll;
    const int p0 = static_cast<int>(min(static_cast<int64_t>(me) * each, static_cast<int64_t>(a.num_pages)));
    const int p1 = min(p0 + each, a.num_pages);
    int64_t rank = 0, have = 0;
    if (code == 0 && want > 0) {  // (every CTA comes to the same verdict and count)
        int64_t free_pages = 0;
        for (int p = p0; p < p1; ++p) free_pages += a.refs[p] == 0;
        rank = cluster_scan(free_pages, sh, 0, have);  // also: every CTA has read lens, table and refs
        if (have < want) code = kNoPages;
    }
    if (me == 0) {
        a.info[0] = code;
        a.info[1] = code < 0 ? 0 : static_cast<int>(want);
        if (a.n > 0) a.pairs[0] = code < 0 ? 0 : copies;
    }
    if (code == 0 && want > 0)
        for (int p = p0; p < p1 && rank < want; ++p) {
            if (a.refs[p] != 0) continue;
            const int i = owner(sh.need, a.n, static_cast<int>(rank)), k = static_cast<int>(rank) - sh.need[i];
            const int s = a.seqs[i], len = a.lens[s], copy = sh.copy[i];
            int* at = a.table + s * a.table_stride + (copy != kNoCopy ? len / a.page_size : pages_for(len, a.page_size)) + k;
            if (copy != kNoCopy && k == 0) {
                a.pairs[1 + 2 * copy] = *at;
                a.pairs[2 + 2 * copy] = p;
            }
            *at = p;
            a.refs[p] = 1;  // only this thread looks at p
            ++rank;
        }
    cl.sync();
    if (cl.block_rank() != 0) return;  // what is left is short: one CTA, so that its own barrier orders it
    if (code < 0) {
        for (int i = threadIdx.x; i < (a.slots ? a.slots_cap : 0); i += kThreads) a.slots[i] = -1;
        return;
    }
    // a copied page loses a holder, only now that no thread looks for free pages any more
    for (int i = threadIdx.x; i < copies; i += kThreads) atomicSub(&a.refs[a.pairs[1 + 2 * i]], 1);
    for (int i = threadIdx.x; i < (a.slots ? a.slots_cap : 0); i += kThreads) {
        int slot = -1;
        if (i < tokens) {
            const int o = owner(sh.add, a.n, i), s = a.seqs[o], pos = a.lens[s] + i - sh.add[o];
            slot = a.table[s * a.table_stride + pos / a.page_size] * a.page_size + pos % a.page_size;
        }
        a.slots[i] = slot;
    }
    __syncthreads();  // lengths change once nobody reads them any more
    for (int i = threadIdx.x; i < a.n; i += kThreads) a.lens[a.seqs[i]] += a.other[i];
}

// Pages in use behind the first `live` move into the holes among those: the i-th such page into the
// i-th hole.  pairs[0] = moves, then (source, destination); map[p] = new place of page p >= live.
__global__ void __cluster_dims__(kCluster) __launch_bounds__(kThreads) kv_compact_kernel(const KvPagesArgs a, int* map) {
    __shared__ Shared sh;
    cg::cluster_group cl = cg::this_cluster();
    pdl_launch_dependents();
    pdl_wait();
    const int me = cl.block_rank() * kThreads + threadIdx.x;
    const int each = (a.num_pages + kAll - 1) / kAll;
    const int p0 = static_cast<int>(min(static_cast<int64_t>(me) * each, static_cast<int64_t>(a.num_pages)));
    const int p1 = min(p0 + each, a.num_pages);
    int64_t n = 0, live;
    for (int p = p0; p < p1; ++p) n += a.refs[p] > 0;
    cluster_scan(n, sh, 0, live);
    int64_t movers = 0, holes = 0;
    for (int p = p0; p < p1; ++p) {
        const bool used = a.refs[p] > 0;
        movers += used && p >= live;
        holes += !used && p < live;
    }
    int64_t moves;
    int64_t at = cluster_scan(movers << 32 | holes, sh, 1, moves);
    int src = static_cast<int>(at >> 32), dst = static_cast<int>(at & 0xffffffff);
    for (int p = p0; p < p1; ++p) {
        const bool used = a.refs[p] > 0;
        if (used && p >= live) a.pairs[1 + 2 * src++] = p;
        if (!used && p < live) a.pairs[2 + 2 * dst++] = p;
        if (p >= live) map[p] = p;
    }
    const int count = static_cast<int>(moves & 0xffffffff);
    if (me == 0) {
        a.pairs[0] = count;
        a.info[0] = 0;
        a.info[1] = static_cast<int>(live);
    }
    cl.sync();
    for (int i = me; i < count; i += kAll) {
        const int from = a.pairs[1 + 2 * i], to = a.pairs[2 + 2 * i];
        map[from] = to;
        a.refs[to] = a.refs[from];
        a.refs[from] = 0;
    }
}

// Copies pages pairs[1 + 2 i] -> pairs[2 + 2 i] in every layer, and (compaction) rewrites the block
// tables.  HBM-bound: 16-byte loads, four in flight a thread; a block takes a chunk of one page at a time.
constexpr int kCopyThreads = 256;
constexpr int kChunk = kCopyThreads * 16 * 4;

template <bool REMAP>
__global__ void __launch_bounds__(kCopyThreads)
    kv_move_kernel(const KvPagesArgs a, uint8_t* cache, int64_t layers, int64_t layer_stride, int64_t page_bytes,
                   const int* map) {
    pdl_launch_dependents();
    pdl_wait();
    if constexpr (REMAP) {
        const int live = a.info[1];
        const int64_t cells = static_cast<int64_t>(a.max_seqs) * a.max_pages;
        for (int64_t i = blockIdx.x * int64_t(kCopyThreads) + threadIdx.x; i < cells; i += int64_t(gridDim.x) * kCopyThreads) {
            const int s = static_cast<int>(i / a.max_pages), k = static_cast<int>(i % a.max_pages);
            if (static_cast<int64_t>(k) * a.page_size >= a.lens[s]) continue;
            int* at = a.table + s * a.table_stride + k;
            const int pg = *at;
            if (pg >= live && pg < a.num_pages) *at = map[pg];
        }
    }
    const int64_t chunks = (page_bytes + kChunk - 1) / kChunk;
    const int64_t items = a.pairs[0] * layers * chunks;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t c = it % chunks, rest = it / chunks, l = rest % layers, i = rest / layers;
        const uint8_t* src = cache + l * layer_stride + a.pairs[1 + 2 * i] * page_bytes;
        uint8_t* dst = cache + l * layer_stride + a.pairs[2 + 2 * i] * page_bytes;
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t o = c * kChunk + (k * kCopyThreads + threadIdx.x) * 16;
            if (o < page_bytes) v[k] = *reinterpret_cast<const uint4*>(src + o);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int64_t o = c * kChunk + (k * kCopyThreads + threadIdx.x) * 16;
            if (o < page_bytes) *reinterpret_cast<uint4*>(dst + o) = v[k];
        }
    }
}

template <typename K, typename... A>
int launch(K kernel, int grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

int move_grid(int64_t most, int64_t layers, int64_t page_bytes) {
    const int64_t items = most * layers * ceil_div(page_bytes, kChunk), full = int64_t(sm_count()) * 8;
    return static_cast<int>(items < full ? (items > 0 ? items : 1) : full);
}

}  // namespace

int launch_kv_fork(const KvPagesArgs& a, cudaStream_t st) { return launch(kv_fork_kernel, kCluster, kThreads, 0, st, a, status_ptr()); }

int launch_kv_truncate(const KvPagesArgs& a, cudaStream_t st) {
    return launch(kv_truncate_kernel, kCluster, kThreads, 0, st, a, status_ptr());
}

int launch_kv_reserve(const KvPagesArgs& a, uint8_t* cache, int64_t layers, int64_t layer_stride, int64_t page_bytes,
                      cudaStream_t st) {
    static std::atomic<int> known[64];  // devices that allow the kernel its shared memory
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ERR_CUDA;
    if (known[dev].load() == 0) {
        if (cudaFuncSetAttribute(kv_reserve_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Reserve)) != cudaSuccess)
            return MXQ_ERR_CUDA;
        known[dev].store(1);
    }
    const int rc = launch(kv_reserve_kernel, kCluster, kThreads, sizeof(Reserve), st, a);
    if (rc != MXQ_OK || a.n == 0) return rc;
    return launch(kv_move_kernel<false>, move_grid(a.n, layers, page_bytes), kCopyThreads, 0, st, a, cache, layers, layer_stride,
                  page_bytes, static_cast<const int*>(nullptr));
}

int launch_kv_compact(const KvPagesArgs& a, uint8_t* cache, int64_t layers, int64_t layer_stride, int64_t page_bytes,
                      cudaStream_t st) {
    int* map = a.pairs + 1 + 2 * static_cast<int64_t>(a.num_pages);
    const int rc = launch(kv_compact_kernel, kCluster, kThreads, 0, st, a, map);
    if (rc != MXQ_OK) return rc;
    return launch(kv_move_kernel<true>, sm_count() * 8, kCopyThreads, 0, st, a, cache, layers, layer_stride, page_bytes,
                  static_cast<const int*>(map));
}

}  // namespace mxq
