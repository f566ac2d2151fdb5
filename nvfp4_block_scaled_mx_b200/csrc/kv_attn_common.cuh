// kv_attn_common.cuh -- what the two attention kernels over the 4-bit cache share: a sequence and its
// spans, the even cut of a batch's work, instructions, and the kernel that joins parts of row tiles.
#pragma once

#include "kv.cuh"
#include "kv_internal.h"

namespace mxq {
namespace {

constexpr float kNegMax = -3.402823466e38f;
constexpr int kMaxGrid = 1024;  // CTAs of one launch, as many as the join kernel's list holds

// A run of token tiles of one row tile and kv head, as the feeding warp describes it.
struct Segment {
    int count;                     // token tiles; -1: no more work
    uint32_t base;                 // tiles in front of it in the CTA's ring
    int pos0;                      // first token of its first tile
    int seen0, seen1, all0, all1;  // tokens that any row sees, and that all rows see
    int q0, row0, rows, head;      // first query row of the sequence, row tile, its rows, kv head
    int kv, qn;                    // of the sequence: tokens, query rows
    int begins, whole;             // has the row tile's first token tile; has all of them
    int parts;                     // if it begins but is not whole: CTAs that have a part
};

// One sequence as the kernels see it.
struct Seq {
    int kv, q0, qn;  // tokens in the cache, first query row, query rows
};

__device__ __noinline__ Seq load_seq(const KvAttnArgs& a, int b) {
    // all loads first: one round trip
    const bool given = a.q_start != nullptr;
    const int kv = a.lens[b], q0 = given ? a.q_start[b] : b * a.max_q, q1 = given ? a.q_start[b + 1] : q0 + a.max_q;
    Seq s;
    s.kv = min(max(kv, 0), a.max_len);
    s.q0 = q0;
    s.qn = max(q1 - q0, 0);
    const bool bad_rows = q0 < 0 || q1 < q0 || q1 > a.rows_total || s.qn > a.max_q;
    if (bad_rows) s.q0 = s.qn = 0;
    if (bad_rows || kv > a.max_len) kv_status(a.status, bad_rows ? kStatusKvRows : kStatusKvLen);
    return s;
}

// Tokens [first, end) that row r of the sequence sees.
__device__ __forceinline__ void row_span(const KvAttnArgs& a, const Seq& s, int r, int& first, int& end) {
    const int seen = s.kv - s.qn + (a.max_q == 1 ? 0 : r / a.group) + 1;
    end = a.causal ? max(seen, 0) : s.kv;
    first = a.window > 0 ? max(seen - a.window, 0) : 0;
}

// Token tiles [first, first + count) of a row tile; an empty one counts as one tile, so that its rows are
// written.  Out of line, like what else runs once per segment: this code comes from a cold instruction
// cache, and its size was most of a small call's time.
struct TileSpan {
    int first, count;
};
template <int TILE, int ROWS>
__device__ __noinline__ TileSpan tile_span(const KvAttnArgs& a, int kv, int qn, int qt) {
    Seq s;
    s.kv = kv, s.q0 = 0, s.qn = qn;
    const int rows = qn * a.group, r0 = qt * ROWS, r1 = min(r0 + ROWS, rows) - 1;
    int first, end, skip;
    row_span(a, s, r0, first, end);
    if (a.max_q > 1) row_span(a, s, r1, skip, end);  // (the rows of one query token see the same)
    TileSpan t;
    t.first = first / TILE;
    t.count = max((end + TILE - 1) / TILE - t.first, 1);
    return t;
}

// Work of a sequence in token tiles.  A row tile counts EXTRA tiles in front of its own: what a CTA takes to
// begin one (without them the CTAs with many short sequences ended last, 14 of 50 us behind the median).
template <int TILE, int ROWS, int EXTRA>
__device__ __noinline__ int64_t seq_cost(const KvAttnArgs& a, int kv, int qn) {
    int64_t n = 0;
    const int tiles = (qn * a.group + ROWS - 1) / ROWS;
#pragma unroll 1
    for (int qt = 0; qt < tiles; ++qt) n += tile_span<TILE, ROWS>(a, kv, qn, qt).count + EXTRA;
    return n * a.kv_heads;
}

// Inclusive sum over the warp's lanes.
__device__ __noinline__ int64_t warp_scan(int64_t v) {
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += x;
    }
    return v;
}

// The same as seq_cost by the whole warp, 32 row tiles at once; and the row tile that holds place `off` of it, which
// becomes the place in that row tile.  (For a chunk of 700 tokens of 5 heads a lane's own 28 steps took 9 us.)
struct Place {
    int64_t off;  // (or the whole work, for a place behind it)
    int qt;
};
template <int TILE, int ROWS, int EXTRA>
__device__ __noinline__ Place seq_cost_warp(const KvAttnArgs& a, int kv, int qn, int64_t off) {
    const int lane = threadIdx.x & 31, tiles = (qn * a.group + ROWS - 1) / ROWS;
    int64_t before = 0;
#pragma unroll 1
    for (int q0 = 0; q0 < tiles; q0 += 32) {
        const int64_t mine = q0 + lane < tiles ? static_cast<int64_t>(tile_span<TILE, ROWS>(a, kv, qn, q0 + lane).count + EXTRA) * a.kv_heads : 0;
        __syncwarp();
        const int64_t upto = before + warp_scan(mine);
        const uint32_t hit = __ballot_sync(0xffffffffu, upto > off);
        if (hit) {
            const int l = __ffs(hit) - 1;
            return {off - __shfl_sync(0xffffffffu, upto - mine, l), q0 + l};
        }
        before = __shfl_sync(0xffffffffu, upto, 31);
    }
    return {before, tiles};
}

// A lane's sequence's work, for all lanes: row tiles by the sequences' lanes, or by the whole warp where that is
// fewer steps.
template <int TILE, int ROWS, int EXTRA>
__device__ __noinline__ int64_t seq_costs(const KvAttnArgs& a, int kv, int qn) {
    const int lane = threadIdx.x & 31, tiles = (qn * a.group + ROWS - 1) / ROWS;
    uint32_t many = __ballot_sync(0xffffffffu, tiles > 1);
    if (__reduce_max_sync(0xffffffffu, tiles) <= 2 * __popc(many)) many = 0;
    int64_t own = many >> lane & 1u ? 0 : seq_cost<TILE, ROWS, EXTRA>(a, kv, qn);
    __syncwarp();
#pragma unroll 1
    for (; many; many &= many - 1) {
        const int l = __ffs(many) - 1;
        const int64_t n = seq_cost_warp<TILE, ROWS, EXTRA>(a, __shfl_sync(0xffffffffu, kv, l), __shfl_sync(0xffffffffu, qn, l), INT64_MAX).off;
        if (lane == l) own = n;
    }
    return own;
}

// n / d for quotients below 2^20: a float quotient, corrected by at most a step or two (a 64-bit division
// is many more instructions, and this code runs once per segment from a cold instruction cache).
__device__ __forceinline__ int div_small(int64_t n, int64_t d, int64_t& r) {
    int q = static_cast<int>(__fdividef(static_cast<float>(n), static_cast<float>(d)));
    r = n - q * d;
    while (r < 0) r += d, --q;
    while (r >= d) r -= d, ++q;
    return q;
}

// The cut of the batch's work, in token tiles: CTA c takes [c per, (c + 1) per).  Whole warp, every warp
// for itself; `at` is this CTA's first tile, b and qt the sequence and row tile that hold it, off its place there.
struct Plan {
    int64_t work, per, at, off;
    int b, qt;
    Seq s;  // sequence b
};

template <int TILE, int ROWS, int EXTRA>
__device__ __forceinline__ Plan make_plan(const KvAttnArgs& a, int min_tiles) {
    const int lane = threadIdx.x & 31;
    Plan p;
    // of the last 32 sequences: the lane's, its work, and the inclusive sum over the lanes
    Seq s = {};
    int64_t own = 0, sum = 0;
    p.work = 0;
    p.at = 0;
    p.s = s;
    bool locate = false;
    const bool tiled = a.max_q * a.group > ROWS;  // sequences may have more than one row tile
    int64_t base = 0;
#pragma unroll 1
    for (int b0 = 0;; b0 += 32) {  // once for the sum, and again (for more than 32 sequences) to find the place
        if (b0 >= a.batch) {
            if (locate) return p;  // (never: the place lies in front of the end)
            // any share that covers the work will do: the quotient in floats, rounded up past its error of 2^-22
            p.per = static_cast<int64_t>(static_cast<float>(p.work) * a.inv_grid * 1.000001f) + 1;
            if (p.per < min_tiles) p.per = min_tiles;
            p.at = p.per * blockIdx.x;
            p.b = a.batch;
            p.qt = 0;
            p.off = 0;
            if (p.at >= p.work) return p;
            locate = true;
            b0 = a.batch > 32 ? 0 : b0 - 32;
        }
        if (!locate || a.batch > 32) {
            s = {};
            own = 0;
            if (b0 + lane < a.batch) s = load_seq(a, b0 + lane);
            __syncwarp();
            if (tiled)
                own = seq_costs<TILE, ROWS, EXTRA>(a, s.kv, s.qn);
            else if (b0 + lane < a.batch)
                own = seq_cost<TILE, ROWS, EXTRA>(a, s.kv, s.qn);
            __syncwarp();
            sum = warp_scan(own);
        }
        const int64_t all = __shfl_sync(0xffffffffu, sum, 31);
        if (!locate) {
            p.work += all;
            continue;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, base + sum > p.at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            p.off = p.at - base - __shfl_sync(0xffffffffu, sum - own, l);
            p.b = b0 + l;
            p.s.kv = __shfl_sync(0xffffffffu, s.kv, l);
            p.s.q0 = __shfl_sync(0xffffffffu, s.q0, l);
            p.s.qn = __shfl_sync(0xffffffffu, s.qn, l);
            if (tiled) {
                const Place at = seq_cost_warp<TILE, ROWS, EXTRA>(a, p.s.kv, p.s.qn, p.off);
                p.off = at.off, p.qt = at.qt;
            }
            return p;
        }
        base += all;
    }
}

// What the join kernel needs to know of a row tile whose first part CTA c has; parts = 0: there is none.
struct Split {
    int parts, q0, row0, rows, head, pad[3];
};

// ------------------------------------------------------------------------------ instructions

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// 8 E2M1 codes as 4 f16x2: byte i of w becomes o[i], its low nibble in the low half.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&o)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
        : "r"(w));
}

__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t h) {
    uint32_t r;
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(h));
    return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t cvt_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Large scores on tcgen05.  An exponent is fma(s, c, -base), and the base a row's rounded maximum less a few units.  From
// |base| = 2^22 on, a step of fp32 is half a unit and more: what the product is rounded by then parts tokens of one score
// from their own maximum, and what the base is rounded by lets exponents pass what P's f16 takes.  Such rows take
// the branch that raises bases for every tile, where their exponents are rounded products less the base.  There exponents are
// held at the limit, too: all tokens of one score weigh the same, whatever its size.
__device__ __forceinline__ bool far_base(float base) {  // (a row that has seen no token is none)
    return (__float_as_uint(base) & 0x7FFFFFFFu) - 0x4A800000u < 0x7F7FFFFFu - 0x4A800000u;
}
__device__ __forceinline__ float at_most(float x, float top) {  // (NaN stays)
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(top));
    return r;
}

// N bytes (4, 8 or 16) of shared memory as words.
template <int N>
__device__ __forceinline__ void lds(uint32_t addr, uint32_t (&r)[N / 4]) {
    if constexpr (N == 4) {
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r[0]) : "r"(addr));
    } else if constexpr (N == 8) {
        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
    } else {
        static_assert(N == 16, "bytes");
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr));
    }
}

// 2^e as fp32 for e in [-252, 127], as a product of two normal factors where one would not do.
__device__ __forceinline__ float scale_pow2(float x, int e) {
    if (e < -126) {
        x *= __uint_as_float(1u << 23);  // 2^-126
        e += 126;
    }
    return x * __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
}

// mbar_wait_warp with the waiting loop out of line: there are many waits, and their code counts.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, int* status, int where) {
    return mbar_wait(bar, parity, status, where);
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* status, int where) {
    bool ok = mbar_try_wait(bar, parity);
    if (!__all_sync(0xffffffffu, ok)) ok = __all_sync(0xffffffffu, wait_slow(bar, parity, status, where));
    else ok = true;
    return ok;
}

// Mask of the scale bytes of tokens pos (even bytes) and pos + 1 that lie in [first, end).
__device__ __forceinline__ uint32_t pair_mask(int pos, int first, int end) {
    return (pos >= first && pos < end ? 0x00FF00FFu : 0u) | (pos + 1 >= first && pos + 1 < end ? 0xFF00FF00u : 0u);
}

// Writes two, four neighbouring channels of a row.
__device__ __forceinline__ void put2(const KvAttnArgs& a, int64_t at, float x, float y) {
    if (a.out_f32)
        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(x, y);
    else
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at) = __floats2bfloat162_rn(x, y);
}
__device__ __forceinline__ void put4(const KvAttnArgs& a, int64_t at, float x, float y, float z, float w) {
    if (a.out_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + at) = make_float4(x, y, z, w);
    } else {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(x, y), hi = __floats2bfloat162_rn(z, w);
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + at) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
}

// Eight channels.
__device__ __forceinline__ void put8(const KvAttnArgs& a, int64_t at, const float* x) {
    if (a.out_f32) {
        put4(a, at, x[0], x[1], x[2], x[3]);
        put4(a, at + 4, x[4], x[5], x[6], x[7]);
    } else {
        uint32_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            h[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at) = make_uint4(h[0], h[1], h[2], h[3]);
    }
}

// Joins the parts of the row tiles that several CTAs worked on, in CTA order.  Every block gathers the
// list of those from all CTAs' notes; its items are (row tile, slice of 16 channels).  Latency is all
// there is to it: the parts of an item are split among PG groups of threads, each of which has the loads
// of BATCH parts in flight, so that 56 parts (a batch of one on all SMs) take one round trip.
constexpr int kJoinThreads = 256;

// Adds (m2, l2, v2) to the running (m, l, v): sums relative to 2^m.
__device__ __forceinline__ void join_add(float& m, float& l, float4& v, float m2, float l2, const float4& v2) {
    const float top = fmaxf(m, m2), f = ex2(m - top), f2 = ex2(m2 - top);
    m = top;
    l = l * f + l2 * f2;
    v.x = v.x * f + v2.x * f2;
    v.y = v.y * f + v2.y * f2;
    v.z = v.z * f + v2.z * f2;
    v.w = v.w * f + v2.w * f2;
}

template <int FMT, int D, int ROWS>
__global__ void __launch_bounds__(kJoinThreads) kv_attention_join_kernel(const __grid_constant__ KvAttnArgs a, int grid) {
    // a row tile of few parts is one item of all channels; of more, SLICES items
    constexpr int SLICE = ROWS > 64 ? 8 : 16, SLICES = D / SLICE, ELEMS = ROWS * SLICE / 4, PG = kJoinThreads / ELEMS, BATCH = 8;
    constexpr int FEW = ROWS > 64 ? 0 : 4;
    // Parts of 128 rows lie channel by channel (their threads had a row each), smaller ones row by row.
    constexpr bool TRANSPOSED = ROWS == 128;
    constexpr int PART = ROWS * (D + 2);
    __shared__ uint32_t has[2][kMaxGrid / 32];
    __shared__ int list[2][kMaxGrid], count[2];  // [0] of few parts, [1] of more
    __shared__ float2 mls[PG][ELEMS];
    __shared__ float4 vs[PG][ELEMS];
    pdl_launch_dependents();
    pdl_wait();
    const Split* splits = reinterpret_cast<const Split*>(a.partial);
    const float* partials = a.partial + grid * (sizeof(Split) / 4);
    const float gv = FMT == MXQ_NVFP4 ? *a.g_v : 1.0f;
    // the lists are the same in every block: CTAs in order, placed by counting those in front
    int parts[kMaxGrid / kJoinThreads];
#pragma unroll
    for (int i = 0; i < kMaxGrid / kJoinThreads; ++i) {
        const int c = i * kJoinThreads + threadIdx.x;
        parts[i] = c < grid ? splits[c].parts : 0;
    }
#pragma unroll
    for (int i = 0; i < kMaxGrid / kJoinThreads; ++i) {
        const uint32_t m = __ballot_sync(0xffffffffu, parts[i] != 0 && parts[i] <= FEW);
        const uint32_t n = __ballot_sync(0xffffffffu, parts[i] > FEW);
        if ((threadIdx.x & 31) == 0) {
            has[0][(i * kJoinThreads + threadIdx.x) / 32] = m;
            has[1][(i * kJoinThreads + threadIdx.x) / 32] = n;
        }
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        static_assert(kMaxGrid == 32 * 32, "one word of the mask a lane");
        const int which = threadIdx.x >> 5, lane = threadIdx.x & 31;
        uint32_t m = has[which][lane];
        int before = __popc(m);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += x;
        }
        if (lane == 31) count[which] = before;
        before -= __popc(m);
        for (; m; m &= m - 1) list[which][before++] = lane * 32 + __ffs(m) - 1;
    }
    __syncthreads();
    // four channels of row r of all parts k = from, from + step, ...
    auto gather = [&](const float* first, int count, int r, int d, int from, int step, float& m, float& l, float4& v) {
#pragma unroll 1
        for (int k0 = from; k0 < count; k0 += step * BATCH) {
            float2 z[BATCH];
            float4 x[BATCH];
#pragma unroll
            for (int j = 0; j < BATCH; ++j) {
                const int k = k0 + j * step;
                const float* at = first + (k == 0 ? 0 : (2 * k - 1) * static_cast<int64_t>(PART));
                z[j] = make_float2(kNegMax, 0.0f);
                x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (k < count) {
                    z[j] = *reinterpret_cast<const float2*>(at + ROWS * D + 2 * r);
                    if constexpr (TRANSPOSED)
                        x[j] = make_float4(at[d * ROWS + r], at[(d + 1) * ROWS + r], at[(d + 2) * ROWS + r], at[(d + 3) * ROWS + r]);
                    else
                        x[j] = *reinterpret_cast<const float4*>(at + r * D + d);
                }
            }
#pragma unroll
            for (int j = 0; j < BATCH; ++j) join_add(m, l, v, z[j].x, z[j].y, x[j]);
        }
    };
    auto store = [&](const Split& s, int r, int d, float m, float l, const float4& v) {
        const int row = s.row0 + r, j = a.max_q == 1 ? 0 : row / a.group;
        const int64_t o = static_cast<int64_t>(s.q0 + j) * a.heads + s.head * a.group + row - j * a.group;
        const float inv = gv * (l > 0.0f ? 1.0f / l : l);  // l is 0 (no token) or not a number
        put4(a, o * D + d, v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        if (a.lse && d == 0) a.lse[o] = l == 0.0f ? __int_as_float(0xff800000) : (m + log2f(l)) * 0.6931471805599453f;
    };
#pragma unroll 1
    for (int i = blockIdx.x; i < count[0]; i += gridDim.x) {
        const int c = list[0][i];
        const Split s = splits[c];
        // slot 1 of the first CTA, slot 0 of the others
        const float* first = partials + (static_cast<int64_t>(c) * 2 + 1) * PART;
#pragma unroll 1
        for (int e = threadIdx.x; e < ROWS * D / 4; e += kJoinThreads) {
            const int r = TRANSPOSED ? e % ROWS : e / (D / 4), d = (TRANSPOSED ? e / ROWS : e % (D / 4)) * 4;
            if (r >= s.rows) continue;
            float m = kNegMax, l = 0.0f;
            float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < (FEW > 0 ? FEW : 1); ++k) {
                const float* at = first + (k == 0 ? 0 : (2 * k - 1) * static_cast<int64_t>(PART));
                if (k < s.parts) {
                    const float2 z = *reinterpret_cast<const float2*>(at + ROWS * D + 2 * r);
                    float4 x;
                    if constexpr (TRANSPOSED)
                        x = make_float4(at[d * ROWS + r], at[(d + 1) * ROWS + r], at[(d + 2) * ROWS + r], at[(d + 3) * ROWS + r]);
                    else
                        x = *reinterpret_cast<const float4*>(at + r * D + d);
                    join_add(m, l, v, z.x, z.y, x);
                }
            }
            store(s, r, d, m, l, v);
        }
    }
    const int pg = threadIdx.x / ELEMS, e = threadIdx.x % ELEMS;
    const int r = TRANSPOSED ? e % ROWS : e / (SLICE / 4), e4 = TRANSPOSED ? e / ROWS : e % (SLICE / 4);
#pragma unroll 1
    for (int i = blockIdx.x; i < count[1] * SLICES; i += gridDim.x) {
        const int c = list[1][i / SLICES], d = i % SLICES * SLICE + e4 * 4;
        const Split s = splits[c];
        const float* first = partials + (static_cast<int64_t>(c) * 2 + 1) * PART;
        float m = kNegMax, l = 0.0f;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (pg < PG) gather(first, s.parts, r, d, pg, PG, m, l, v);  // (ELEMS need not divide the threads)
        if (pg < PG) {
            mls[pg][e] = make_float2(m, l);
            vs[pg][e] = v;
        }
        __syncthreads();
        if (pg == 0 && r < s.rows) {
#pragma unroll
            for (int k = 1; k < PG; ++k) join_add(m, l, v, mls[k][e].x, mls[k][e].y, vs[k][e]);
            store(s, r, d, m, l, v);
        }
        __syncthreads();
    }
}

}  // namespace
}  // namespace mxq
