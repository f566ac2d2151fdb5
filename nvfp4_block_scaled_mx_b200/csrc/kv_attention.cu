// kv_attention.cu -- attention over the paged 4-bit key/value cache.
//
// One row tile is 8 NT rows (query token x query head of one kv head's group).  A warp turns a tile
// of cached tokens into matrix-instruction operands in registers and keeps its own running softmax:
//   S^T = K Q^T      m16n8k16, f16 x f16 -> fp32: tokens on M, rows on N, so that a group of up to
//                    eight rows wastes nothing and a decoded K operand serves all rows;
//   P   = 2^(s - m)  fp32; m is the warp's running maximum (log2 domain), raised only when a tile exceeds it;
//   O^T = V^T P^T    head channels on M, tokens on K.
// E2M1 codes convert to f16 exactly.  K: NVFP4 codes times their E4M3 scale are exact in f16 (six
// significant bits, at most 2688); MXFP4's power-of-two scale multiplies the fp32 product of its
// 32-element block.  Q is bf16 times a power of two per row (largest element in [2^7, 2^8)), exact in
// f16 but for elements 2^-24 below the row's largest.  V: the scale multiplies P instead of the codes,
// in f16: P is rounded to 11 bits (a bf16 P, 8 bits, would add as much error as the bf16 output has),
// times 2^7 (NVFP4) or 2^4 (MXFP4) so that small probabilities keep their bits.  MXFP4 scales are taken
// relative to the largest one met so far in the same 32 channels; blocks 2^23 below it vanish.
// Sums, maxima and accumulators are fp32.
//
// Work is the list of all (sequence, row tile, kv head, token tile), cut evenly over the CTAs by every
// CTA for itself from the lengths on the device, so that ragged batches balance and a graph can be
// replayed with other lengths.  A CTA's part of a row tile that it does not have whole goes to the
// workspace as (m, l, O); a second kernel joins those in CTA order, so results do not depend on timing.
#include <atomic>

#include "kv.cuh"
#include "kv_internal.h"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMinTiles = 8;  // token tiles a CTA gets at least
constexpr float kNegMax = -3.402823466e38f;

template <int FMT, int D, int NT>
struct Cfg {
    using U = KvUnit<FMT, D>;
    static constexpr int TU = D <= 128 ? 2 : 1;  // units of a token tile
    static constexpr int TILE = 16 * TU;
    static constexpr int ROWS = 8 * NT;
    static constexpr int KS = D / 16;  // k steps of S, m tiles of O
    static constexpr int TILE_BYTES = TU * U::BYTES;
    static constexpr int STAGES = 3;
    static constexpr int RING = kWarps * STAGES * TILE_BYTES;
    static constexpr int OSTRIDE = D + 8;  // floats; row pairs of a warp's float2 stores meet different banks
    static constexpr int RED = kWarps * ROWS * OSTRIDE * 4;
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_RING = NT * KS * 32 * 8;
    static constexpr int OFF_ROW = OFF_RING + (RING > RED ? RING : RED);  // per row: scale, first, end
    static constexpr int OFF_ML = OFF_ROW + ROWS * 12;
    static constexpr int OFF_BAR = (OFF_ML + kWarps * ROWS * 8 + 15) / 16 * 16;
    static constexpr int BYTES = OFF_BAR + kWarps * STAGES * 8 + 64;
    static constexpr float SHIFT = FMT == MXQ_NVFP4 ? 7.0f : 4.0f;  // log2 of what P is multiplied by
};

// One sequence as the kernels see it.
struct Seq {
    int kv, q0, qn;  // tokens in the cache, first query row, query rows
};

__device__ __forceinline__ Seq load_seq(const KvAttnArgs& a, int b) {
    Seq s;
    s.kv = a.lens[b];
    if (s.kv > a.max_len) {
        kv_status(a.status, kStatusKvLen);
        s.kv = a.max_len;
    }
    s.kv = max(s.kv, 0);
    if (a.q_start) {
        const int q0 = a.q_start[b], q1 = a.q_start[b + 1];
        s.q0 = q0;
        s.qn = max(q1 - q0, 0);
        if (q0 < 0 || q1 > a.rows_total || s.qn > a.max_q) {
            kv_status(a.status, kStatusKvRows);
            s.q0 = s.qn = 0;
        }
    } else {
        s.q0 = b * a.max_q;
        s.qn = a.max_q;
    }
    return s;
}

// Tokens [first, end) that row r of the sequence sees.
__device__ __forceinline__ void row_span(const KvAttnArgs& a, const Seq& s, int r, int& first, int& end) {
    const int seen = s.kv - s.qn + r / a.group + 1;
    end = a.causal ? max(seen, 0) : s.kv;
    first = a.window > 0 ? max(seen - a.window, 0) : 0;
}

// Token tiles [t0, t0 + n) of a row tile; an empty one counts as one tile, so that its rows are written.
template <int TILE, int ROWS>
__device__ __forceinline__ int tile_span(const KvAttnArgs& a, const Seq& s, int qt, int& t0) {
    const int rows = s.qn * a.group, r0 = qt * ROWS, r1 = min(r0 + ROWS, rows) - 1;
    int first, end, skip;
    row_span(a, s, r0, first, skip);
    row_span(a, s, r1, skip, end);
    t0 = first / TILE;
    return max((end + TILE - 1) / TILE - t0, 1);
}

template <int TILE, int ROWS>
__device__ __forceinline__ int64_t seq_cost(const KvAttnArgs& a, const Seq& s) {
    int64_t n = 0;
    const int tiles = (s.qn * a.group + ROWS - 1) / ROWS;
    for (int qt = 0; qt < tiles; ++qt) {
        int t0;
        n += tile_span<TILE, ROWS>(a, s, qt, t0);
    }
    return n * a.kv_heads;
}

__device__ __forceinline__ int64_t warp_sum64(int64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// All work of the batch, in token tiles (whole warp).
template <int TILE, int ROWS>
__device__ __forceinline__ int64_t total_work(const KvAttnArgs& a) {
    int64_t n = 0;
    for (int b = threadIdx.x & 31; b < a.batch; b += 32) n += seq_cost<TILE, ROWS>(a, load_seq(a, b));
    return warp_sum64(n);
}

// The sequence that holds work item `at`, and the work in front of it (whole warp; at < total).
template <int TILE, int ROWS>
__device__ __forceinline__ int find_seq(const KvAttnArgs& a, int64_t at, int64_t& before) {
    const int lane = threadIdx.x & 31;
    int64_t base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int b = b0 + lane;
        const int64_t cost = b < a.batch ? seq_cost<TILE, ROWS>(a, load_seq(a, b)) : 0;
        int64_t sum = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += x;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, base + sum > at);
        if (hit) {
            const int l = __ffs(hit) - 1;
            before = base + __shfl_sync(0xffffffffu, sum - cost, l);
            return b0 + l;
        }
        base += __shfl_sync(0xffffffffu, sum, 31);
    }
    before = base;
    return a.batch;
}

__device__ __forceinline__ int64_t work_ctas(int64_t work, int grid) {
    const int64_t n = (work + kMinTiles - 1) / kMinTiles;
    return n < grid ? (n > 0 ? n : 1) : grid;
}

// ------------------------------------------------------------------------------ instructions

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// --------------------------------------------------------------------------------- warp state

template <int FMT, int D, int NT>
struct Warp {
    using C = Cfg<FMT, D, NT>;
    float o[NT][C::KS][4];
    float m[NT][2], l[NT][2];
    int ref[FMT == MXQ_MXFP4 ? C::U::NB : 1];  // MXFP4: E8M0 code that stands for 2^9 in the factors, per 32 channels
};

template <int FMT, int D, int NT>
__device__ __forceinline__ void warp_reset(Warp<FMT, D, NT>& w) {
    using C = Cfg<FMT, D, NT>;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < C::KS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) w.o[n][j][i] = 0.0f;
        w.m[n][0] = w.m[n][1] = kNegMax;
        w.l[n][0] = w.l[n][1] = 0.0f;
    }
    if constexpr (FMT == MXQ_MXFP4) {
#pragma unroll
        for (int b = 0; b < C::U::NB; ++b) w.ref[b] = -1000;
    }
}

// Scores of one token tile: s[u][n] holds tokens g, g + 8 of unit u for rows 2t, 2t + 1 of n-tile n.
template <int FMT, int D, int NT>
__device__ __forceinline__ void scores(uint32_t tile, uint32_t qf, float (&s)[Cfg<FMT, D, NT>::TU][NT][4]) {
    using C = Cfg<FMT, D, NT>;
    using U = typename C::U;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int u = 0; u < C::TU; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n) s[u][n][0] = s[u][n][1] = s[u][n][2] = s[u][n][3] = 0.0f;

    // scales of tokens g and g + 8: NVFP4 f16x2 (s, s) per 8 bytes of this lane's quarter, MXFP4 fp32 per block
    constexpr int NSC = FMT == MXQ_NVFP4 ? D / 64 : U::NB;
    uint32_t sc[C::TU][2][NSC];
#pragma unroll
    for (int u = 0; u < C::TU; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = tile + u * U::BYTES + U::OFF_KS + (g + 8 * h) * U::NB;
            if constexpr (FMT == MXQ_NVFP4) {
                uint32_t x;
                if constexpr (NSC == 1) {
                    x = ld_shared_u8(at + t);
                } else if constexpr (NSC == 2) {
                    x = ld_shared_u16(at + 2 * t);
                } else {
                    uint32_t r[1];
                    lds<4>(at + 4 * t, r);
                    x = r[0];
                }
#pragma unroll
                for (int i = 0; i < NSC; i += 2) {
                    const uint32_t f = e4m3x2_f16x2(x >> (8 * i));
                    sc[u][h][i] = prmt(f, f, 0x1010u);
                    if (i + 1 < NSC) sc[u][h][i + 1] = prmt(f, f, 0x3232u);
                }
            } else {
                uint32_t x[2] = {0, 0};
                if constexpr (U::NB == 2) {
                    x[0] = ld_shared_u16(at);
                } else if constexpr (U::NB == 4) {
                    uint32_t r[1];
                    lds<4>(at, r);
                    x[0] = r[0];
                } else {
                    lds<8>(at, x);
                }
#pragma unroll
                for (int i = 0; i < NSC; ++i) sc[u][h][i] = (x[i >> 2] >> (8 * (i & 3)) & 0xFFu) << 23;
            }
        }

#pragma unroll
    for (int p = 0; p < U::PIECES; ++p) {
        uint32_t k[C::TU][2][U::W / 4];
#pragma unroll
        for (int u = 0; u < C::TU; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) lds<U::W>(tile + u * U::BYTES + U::k_at(g + 8 * h, t, p * U::W), k[u][h]);
#pragma unroll
        for (int w = 0; w < U::W / 4; ++w) {
            const int word = p * (U::W / 4) + w;  // k steps 2 word, 2 word + 1
            uint32_t q[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n) lds<16>(qf + ((n * (C::KS / 2) + word) * 32 + lane) * 16, q[n]);
#pragma unroll
            for (int u = 0; u < C::TU; ++u) {
                uint32_t lo[4], hi[4];
                e2m1x8(k[u][0][w], lo);
                e2m1x8(k[u][1][w], hi);
                if constexpr (FMT == MXQ_NVFP4) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        lo[i] = hmul2(lo[i], sc[u][0][word / 2]);
                        hi[i] = hmul2(hi[i], sc[u][1][word / 2]);
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_f16(s[u][n], lo[0], hi[0], lo[1], hi[1], q[n][0], q[n][1]);
                        mma_f16(s[u][n], lo[2], hi[2], lo[3], hi[3], q[n][2], q[n][3]);
                    }
                } else {
                    const float f0 = __uint_as_float(sc[u][0][word]), f1 = __uint_as_float(sc[u][1][word]);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        mma_f16(c, lo[0], hi[0], lo[1], hi[1], q[n][0], q[n][1]);
                        mma_f16(c, lo[2], hi[2], lo[3], hi[3], q[n][2], q[n][3]);
                        s[u][n][0] = fmaf(c[0], f0, s[u][n][0]);
                        s[u][n][1] = fmaf(c[1], f0, s[u][n][1]);
                        s[u][n][2] = fmaf(c[2], f1, s[u][n][2]);
                        s[u][n][3] = fmaf(c[3], f1, s[u][n][3]);
                    }
                }
            }
        }
    }
}

// Masks of the f16 pair (tokens pos, pos + 1) for a row that sees [first, end).
__device__ __forceinline__ uint32_t pair_mask(int pos, int first, int end) {
    return (pos >= first && pos < end ? 0x0000FFFFu : 0u) | (pos + 1 >= first && pos + 1 < end ? 0xFFFF0000u : 0u);
}

// One token tile: scores, softmax update, O update.  pos0 is the tile's first token; MASK: some row does
// not see all of its tokens; seen0 / seen1: tokens that any row of the tile sees.
template <int FMT, int D, int NT, bool MASK>
__device__ __forceinline__ void tile_step(Warp<FMT, D, NT>& w, uint32_t tile, uint32_t qf, const float (&cs)[NT][2],
                                          const int* row_first, const int* row_end, int pos0, int seen0, int seen1) {
    using C = Cfg<FMT, D, NT>;
    using U = typename C::U;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float s[C::TU][NT][4];
    scores<FMT, D, NT>(tile, qf, s);

    bool raise = false;
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            int first = 0, end = 0;
            if constexpr (MASK) first = row_first[8 * n + 2 * t + c], end = row_end[8 * n + 2 * t + c];
            float x = kNegMax;
#pragma unroll
            for (int u = 0; u < C::TU; ++u)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float v = s[u][n][2 * h + c] * cs[n][c];
                    if constexpr (MASK) {
                        const int pos = pos0 + 16 * u + 8 * h + g;
                        if (pos < first || pos >= end) v = __int_as_float(0xff800000);
                    }
                    s[u][n][2 * h + c] = v;
                    x = fmaxf(x, v);
                }
            top[n][c] = x;
            raise = raise || x > w.m[n][c];
        }
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float al[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = top[n][c];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, off));
                x = fmaxf(x, w.m[n][c]);
                al[c] = ex2(w.m[n][c] - x);
                w.m[n][c] = x;
                w.l[n][c] *= al[c];
            }
#pragma unroll
            for (int j = 0; j < C::KS; ++j) {
                w.o[n][j][0] *= al[0];
                w.o[n][j][1] *= al[1];
                w.o[n][j][2] *= al[0];
                w.o[n][j][3] *= al[1];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < C::TU; ++u) {
        uint32_t p[NT][2];  // rows g of n-tile n; tokens 2t, 2t + 1 of either group of eight
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float e[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) e[i] = ex2(s[u][n][i] - (w.m[n][i & 1] - C::SHIFT));
            w.l[n][0] += e[0] + e[2];
            w.l[n][1] += e[1] + e[3];
            p[n][0] = transpose8x8(cvt_f16x2(e[0], e[1]));
            p[n][1] = transpose8x8(cvt_f16x2(e[2], e[3]));
        }
        uint32_t keep[NT][2];
        uint32_t live[2] = {0xFFFFFFFFu, 0xFFFFFFFFu};  // tokens any row sees
        if constexpr (MASK) {
            const int pos = pos0 + 16 * u + 2 * t;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                live[h] = pair_mask(pos + 8 * h, seen0, seen1);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    keep[n][h] = pair_mask(pos + 8 * h, row_first[8 * n + g], row_end[8 * n + g]);
            }
        }
        const uint32_t unit = tile + u * U::BYTES;
        // scale factors of the pair's two tokens, f16x2 per scale block
        uint32_t fac[2][U::NB];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            constexpr int PB = 2 * U::NB;  // bytes of a token pair's scales
            uint32_t x[PB / 4];
            const uint32_t at = unit + U::OFF_VS + (t + 4 * h) * PB;
            if constexpr (PB <= 16) {
                lds<PB>(at, x);
            } else {
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < PB / 16; ++i) {
                    lds<16>(at + 16 * i, y);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[4 * i + k] = y[k];
                }
            }
#pragma unroll
            for (int b = 0; b < U::NB; ++b) {
                const uint32_t pair = b & 1 ? x[b >> 1] >> 16 : x[b >> 1] & 0xFFFFu;
                if constexpr (FMT == MXQ_NVFP4) {
                    fac[h][b] = e4m3x2_f16x2(pair);
                } else {
                    fac[h][b] = prmt(pair, 0u, 0x4140u);  // the codes, one a half
                    if constexpr (MASK) fac[h][b] &= live[h];
                }
            }
        }
        if constexpr (FMT == MXQ_MXFP4) {
            // factors 2^(code - ref + 9) as f16 bits; a code more than 2 above ref moves ref (and O) up
            bool over = false;
#pragma unroll
            for (int b = 0; b < U::NB; ++b) {
                const uint32_t hi = __vmaxu2(fac[0][b], fac[1][b]);
                over = over || static_cast<int>(max(hi & 0xFFFFu, hi >> 16)) > w.ref[b] + 2;
            }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int b = 0; b < U::NB; ++b) {
                    const uint32_t hi = __vmaxu2(fac[0][b], fac[1][b]);
                    int code = static_cast<int>(max(hi & 0xFFFFu, hi >> 16));
                    code = max(code, __shfl_xor_sync(0xffffffffu, code, 1));
                    code = max(code, __shfl_xor_sync(0xffffffffu, code, 2));
                    if (code > w.ref[b] + 2) {
                        const float f = scale_pow2(1.0f, max(w.ref[b] - code, -252));
                        w.ref[b] = code;
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int j = 2 * b; j < 2 * b + 2; ++j)
#pragma unroll
                                for (int i = 0; i < 4; ++i) w.o[n][j][i] *= f;
                    }
                }
            }
#pragma unroll
            for (int b = 0; b < U::NB; ++b) {
                const uint32_t bias = static_cast<uint32_t>((24 - w.ref[b]) & 0xFFFF) * 0x10001u;
#pragma unroll
                for (int h = 0; h < 2; ++h) fac[h][b] = __viaddmax_s16x2_relu(fac[h][b], bias, 0u) << 10;
            }
        }
        // V codes: this lane's D / 16 bytes of both tokens of either pair
        uint32_t v[2][2][D / 64];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = unit + U::OFF_V + h * (4 * D) + lane * U::W;
            uint32_t y[U::W / 4];
#pragma unroll
            for (int pc = 0; pc < U::PIECES; ++pc) {
                lds<U::W>(at + pc * 32 * U::W, y);
#pragma unroll
                for (int k = 0; k < U::W / 4; ++k) {
                    const int word = pc * (U::W / 4) + k;
                    v[h][word / (D / 64)][word % (D / 64)] = y[k];
                }
            }
        }
#pragma unroll
        for (int wd = 0; wd < D / 64; ++wd) {
            uint32_t a[4][4];  // [operand register][m tile 4 wd + i]
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x = v[h][0][wd], y = v[h][1][wd];
                e2m1x8((x & 0x0F0F0F0Fu) | (y << 4 & 0xF0F0F0F0u), a[2 * h]);
                e2m1x8((x >> 4 & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u), a[2 * h + 1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int j = 4 * wd + i, b = FMT == MXQ_NVFP4 ? j : j / 2;
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    uint32_t b0 = hmul2(p[n][0], fac[0][b]), b1 = hmul2(p[n][1], fac[1][b]);
                    if constexpr (MASK) b0 &= keep[n][0], b1 &= keep[n][1];
                    mma_f16(w.o[n][j], a[0][i], a[1][i], a[2][i], a[3][i], b0, b1);
                }
            }
        }
    }
}

// ------------------------------------------------------------------------------------- kernel

// Writes one row's share: `x` two neighbouring channels.
__device__ __forceinline__ void put2(const KvAttnArgs& a, int64_t at, float x, float y) {
    if (a.out_f32) {
        *reinterpret_cast<float2*>(static_cast<float*>(a.out) + at) = make_float2(x, y);
    } else {
        *reinterpret_cast<__nv_bfloat162*>(static_cast<__nv_bfloat16*>(a.out) + at) = __floats2bfloat162_rn(x, y);
    }
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(kThreads) kv_attention_kernel(const KvAttnArgs a) {
    using C = Cfg<FMT, D, NT>;
    using U = typename C::U;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    float* row_scale = reinterpret_cast<float*>(smem + C::OFF_ROW);
    int* row_first = reinterpret_cast<int*>(row_scale + C::ROWS);
    int* row_end = row_first + C::ROWS;
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
    uint64_t* full = bars + warp * C::STAGES;
    uint8_t* ring = smem + C::OFF_RING + warp * C::STAGES * C::TILE_BYTES;
    const uint32_t qf = smem_u32(smem + C::OFF_Q);

    if (lane == 0) {
        for (int i = 0; i < C::STAGES; ++i) mbar_init(&full[i], 1);
        fence_barrier_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();

    // this CTA's part of the work (every warp for itself: the loads hit the same lines)
    const int64_t work = total_work<C::TILE, C::ROWS>(a);
    const int64_t ctas = work_ctas(work, gridDim.x);
    if (blockIdx.x >= ctas || work == 0) return;
    int64_t at = work * blockIdx.x / ctas;
    const int64_t stop = work * (blockIdx.x + 1) / ctas;
    int64_t before;
    int b = find_seq<C::TILE, C::ROWS>(a, at, before);
    int64_t off = at - before;  // work of the sequence in front of `at`
    Seq s = load_seq(a, b);
    int qt = 0;
    uint32_t used = 0;  // tiles this warp has taken through its ring

    while (at < stop) {
        // the row tile and kv head that hold work item `at`
        int t0, n;
        for (;;) {
            if (qt * C::ROWS >= s.qn * a.group) {
                s = load_seq(a, ++b);
                qt = 0;
                continue;
            }
            n = tile_span<C::TILE, C::ROWS>(a, s, qt, t0);
            if (off < static_cast<int64_t>(n) * a.kv_heads) break;
            off -= static_cast<int64_t>(n) * a.kv_heads;
            ++qt;
        }
        const int head = static_cast<int>(off / n), from = static_cast<int>(off % n);
        const int count = static_cast<int>(min(static_cast<int64_t>(n - from), stop - at));
        const int rows = min(C::ROWS, s.qn * a.group - qt * C::ROWS);
        const bool whole = from == 0 && count == n;
        int seen0, seen1, skip;
        row_span(a, s, qt * C::ROWS, seen0, skip);
        row_span(a, s, qt * C::ROWS + rows - 1, skip, seen1);
        // tokens that all rows see
        int all0, all1;
        row_span(a, s, qt * C::ROWS, skip, all1);
        row_span(a, s, qt * C::ROWS + rows - 1, all0, skip);

        // this warp's tiles: from + warp, + kWarps, ...; lane i holds the page of the i-th unit ahead
        const int mine = count > warp ? (count - warp + kWarps - 1) / kWarps : 0;
        const int first_tile = t0 + from + warp;
        const int units_end = (seen1 + 15) >> 4;  // units behind it are not loaded (their pages may not exist)
        constexpr int AHEAD = 32 / C::TU;         // tiles whose pages one register per lane holds
        auto page_of = [&](int batch) {
            const int i = batch * AHEAD + lane / C::TU;
            const int unit = (first_tile + i * kWarps) * C::TU + lane % C::TU;
            if (i >= mine || unit >= units_end) return -1;
            const int pg = a.table[static_cast<int64_t>(b) * a.table_stride + unit / a.page_units];
            if (pg < 0 || pg >= a.num_pages) {
                kv_status(a.status, kStatusKvPage);
                return -1;
            }
            return pg;
        };
        int pages = page_of(0), pages_next = page_of(1);
        int issued = 0;
        auto issue = [&]() {  // whole warp: start the copy of tile number `issued`
            if (issued >= mine) return;
            if (issued && issued % AHEAD == 0) {
                pages = pages_next;
                pages_next = page_of(issued / AHEAD + 1);
            }
            const uint32_t stage = (used + issued) % C::STAGES;
            uint8_t* dst = ring + stage * C::TILE_BYTES;
            uint32_t bytes = 0;
            int64_t src[C::TU];
#pragma unroll
            for (int u = 0; u < C::TU; ++u) {
                const int pg = __shfl_sync(0xffffffffu, pages, (issued % AHEAD) * C::TU + u);
                const int unit = (first_tile + issued * kWarps) * C::TU + u;
                src[u] = pg < 0 ? -1
                                : (static_cast<int64_t>(pg) * a.kv_heads + head) * a.page_bytes +
                                      static_cast<int64_t>(unit % a.page_units) * U::BYTES;
                bytes += pg < 0 ? 0 : U::BYTES;
            }
            if (elect_one()) {
                mbar_arrive_expect_tx(&full[stage], bytes);
#pragma unroll
                for (int u = 0; u < C::TU; ++u)
                    if (src[u] >= 0) bulk_load(dst + u * U::BYTES, a.cache + src[u], U::BYTES, &full[stage]);
            }
            ++issued;
        };
#pragma unroll
        for (int i = 0; i < C::STAGES; ++i) issue();

        // Q operands: rows as f16 times a power of two
        for (int r = warp; r < C::ROWS; r += kWarps) {
            constexpr int E = D / 32;  // elements of a lane
            uint32_t x[E / 2];
            float big = 0.0f;
#pragma unroll
            for (int i = 0; i < E / 2; ++i) x[i] = 0;
            if (r < rows) {
                const int row = qt * C::ROWS + r;
                const __nv_bfloat16* src = a.q + static_cast<int64_t>(s.q0 + row / a.group) * a.q_token_stride +
                                           static_cast<int64_t>(head * a.group + row % a.group) * a.q_head_stride + lane * E;
#pragma unroll
                for (int i = 0; i < E / 2; ++i) x[i] = reinterpret_cast<const uint32_t*>(src)[i];
            }
#pragma unroll
            for (int i = 0; i < E / 2; ++i)
                big = fmaxf(big, fmaxf(fabsf(__uint_as_float(x[i] << 16)), fabsf(__uint_as_float(x[i] & 0xFFFF0000u))));
#pragma unroll
            for (int o = 16; o; o >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, o));
            const uint32_t ex = max(__float_as_uint(big) >> 23, 8u);
            const float mul = __uint_as_float((261u - ex) << 23);
            uint32_t h[E / 2];
#pragma unroll
            for (int i = 0; i < E / 2; ++i)
                h[i] = cvt_f16x2(__uint_as_float(x[i] << 16) * mul, __uint_as_float(x[i] & 0xFFFF0000u) * mul);
            // element e of the row: lane (r % 8, qq) and k step st, as its A operand's codes are dealt
            const int e = lane * E;
            int qq, st;
            if constexpr (FMT == MXQ_NVFP4) {
                qq = e / (D / 4);
                st = e % (D / 4) / 4;
            } else {
                qq = e % 32 / 8;
                st = 2 * (e / 32) + e % 8 / 4;
            }
            uint32_t* dst = reinterpret_cast<uint32_t*>(
                smem + C::OFF_Q + (((r / 8) * (C::KS / 2) + st / 2) * 32 + (r % 8) * 4 + qq) * 16 + (st & 1) * 8 + e % 4 / 2 * 4);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) dst[i] = h[i];
            if (lane == 0) {
                float f = a.scale * 1.4426950408889634f;
                if constexpr (FMT == MXQ_NVFP4) f *= *a.g_k;
                row_scale[r] = f * __uint_as_float((ex - 7u) << 23);
                int f0 = 0, f1 = 0;
                if (r < rows) row_span(a, s, qt * C::ROWS + r, f0, f1);
                row_first[r] = f0;
                row_end[r] = f1;
            }
        }
        __syncthreads();
        float cs[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) cs[i][c] = row_scale[8 * i + 2 * t + c];

        Warp<FMT, D, NT> w;
        warp_reset(w);
        bool dead = false;
        for (int i = 0; i < mine; ++i) {
            const uint32_t slot = (used + i) % C::STAGES;
            if (!mbar_wait_warp(&full[slot], (used + i) / C::STAGES & 1u, a.status, 0x40)) {
                dead = true;
                break;
            }
            const uint32_t tile = smem_u32(ring + slot * C::TILE_BYTES);
            const int pos0 = (first_tile + i * kWarps) * C::TILE;
            if (pos0 >= all0 && pos0 + C::TILE <= all1)
                tile_step<FMT, D, NT, false>(w, tile, qf, cs, row_first, row_end, pos0, seen0, seen1);
            else
                tile_step<FMT, D, NT, true>(w, tile, qf, cs, row_first, row_end, pos0, seen0, seen1);
            __syncwarp();
            issue();
        }
        used += mine;

        // join the warps: each brings its O to the common maximum, then sums
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = w.l[i][c];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (g == 0) ml[warp * C::ROWS + 8 * i + 2 * t + c] = make_float2(w.m[i][c], x);
            }
        if (__syncthreads_or(dead)) return;
        float* red = reinterpret_cast<float*>(smem + C::OFF_RING);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            float f[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float top = kNegMax;
#pragma unroll
                for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml[k * C::ROWS + 8 * i + 2 * t + c].x);
                f[c] = ex2(w.m[i][c] - top);
            }
#pragma unroll
            for (int j = 0; j < C::KS; ++j) {
                float x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k] = w.o[i][j][k] * f[k & 1];
                    if constexpr (FMT == MXQ_MXFP4) x[k] = scale_pow2(x[k], max(w.ref[j / 2], 0) - 136);
                }
                float* dst = red + (warp * C::ROWS + 8 * i + 2 * t) * C::OSTRIDE + 16 * j + 2 * g;
                *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[2]);
                *reinterpret_cast<float2*>(dst + C::OSTRIDE) = make_float2(x[1], x[3]);
            }
        }
        __syncthreads();
        float* part = a.partial + (static_cast<int64_t>(blockIdx.x) * 2 + (from == 0 ? 1 : 0)) * (C::ROWS * (D + 2));
        for (int i = threadIdx.x; i < C::ROWS * (D / 2); i += kThreads) {
            const int r = i / (D / 2), d = i % (D / 2) * 2;
            float top = kNegMax, sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml[k * C::ROWS + r].x);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float2 z = ml[k * C::ROWS + r];
                sum += z.y * ex2(z.x - top);
                const float2 v = *reinterpret_cast<const float2*>(red + (k * C::ROWS + r) * C::OSTRIDE + d);
                x += v.x;
                y += v.y;
            }
            if (whole) {
                if (r < rows) {
                    const int row = qt * C::ROWS + r;
                    const int64_t o = static_cast<int64_t>(s.q0 + row / a.group) * a.heads + head * a.group + row % a.group;
                    float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
                    if constexpr (FMT == MXQ_NVFP4) inv *= *a.g_v;
                    put2(a, o * D + d, x * inv, y * inv);
                    if (a.lse && d == 0)
                        a.lse[o] = sum == 0.0f ? __int_as_float(0xff800000)
                                               : (top + (log2f(sum) - C::SHIFT)) * 0.6931471805599453f;
                }
            } else {
                *reinterpret_cast<float2*>(part + r * D + d) = make_float2(x, y);
                if (d == 0) *reinterpret_cast<float2*>(part + C::ROWS * D + 2 * r) = make_float2(top, sum);
            }
        }
        fence_proxy_async_smem();  // the ring, written above by plain stores, takes bulk copies again
        __syncthreads();
        at += count;
        off += count;
    }
}

// Joins the parts of the row tiles that several CTAs worked on: block x stands for the cut between CTAs
// x and x + 1 and acts if that is the first cut inside its row tile; y slices the channels.
constexpr int kJoinSlice = 32;
template <int FMT, int D, int NT>
__global__ void __launch_bounds__(256) kv_attention_join_kernel(const KvAttnArgs a, int grid) {
    using C = Cfg<FMT, D, NT>;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t work = total_work<C::TILE, C::ROWS>(a);
    const int64_t ctas = work_ctas(work, grid);
    const int64_t me = blockIdx.x;
    if (me + 1 >= ctas || work == 0) return;
    const int64_t cut = work * (me + 1) / ctas;
    int64_t before;
    const int b = find_seq<C::TILE, C::ROWS>(a, cut, before);
    const Seq s = load_seq(a, b);
    int64_t off = cut - before;
    int qt = 0, n, t0;
    for (;; ++qt) {
        n = tile_span<C::TILE, C::ROWS>(a, s, qt, t0);
        if (off < static_cast<int64_t>(n) * a.kv_heads) break;
        off -= static_cast<int64_t>(n) * a.kv_heads;
    }
    const int head = static_cast<int>(off / n), from = static_cast<int>(off % n);
    if (from == 0) return;                        // the cut lies between two row tiles
    const int64_t begin = cut - from, end = begin + n;
    if (work * me / ctas > begin) return;         // an earlier cut lies in this row tile
    int parts = 1;
    while (work * (me + parts) / ctas < end) ++parts;  // CTAs me .. me + parts - 1 have a part
    const int rows = min(C::ROWS, s.qn * a.group - qt * C::ROWS);
    constexpr int64_t PART = C::ROWS * (D + 2);
    auto part = [&](int k) { return a.partial + ((me + k) * 2 + (k == 0 ? 1 : 0)) * PART; };
    for (int i = threadIdx.x; i < rows * (kJoinSlice / 2); i += 256) {
        const int r = i / (kJoinSlice / 2), d = blockIdx.y * kJoinSlice + i % (kJoinSlice / 2) * 2;
        float top = kNegMax;
#pragma unroll 8
        for (int k = 0; k < parts; ++k) top = fmaxf(top, part(k)[C::ROWS * D + 2 * r]);
        float sum = 0.0f, x = 0.0f, y = 0.0f;
#pragma unroll 8
        for (int k = 0; k < parts; ++k) {
            const float2 z = *reinterpret_cast<const float2*>(part(k) + C::ROWS * D + 2 * r);
            const float2 v = *reinterpret_cast<const float2*>(part(k) + r * D + d);
            const float f = ex2(z.x - top);
            sum += z.y * f;
            x = fmaf(v.x, f, x);
            y = fmaf(v.y, f, y);
        }
        const int row = qt * C::ROWS + r;
        const int64_t o = static_cast<int64_t>(s.q0 + row / a.group) * a.heads + head * a.group + row % a.group;
        float inv = sum > 0.0f ? 1.0f / sum : (sum == 0.0f ? 0.0f : sum);
        if constexpr (FMT == MXQ_NVFP4) inv *= *a.g_v;
        put2(a, o * D + d, x * inv, y * inv);
        if (a.lse && d == 0)
            a.lse[o] = sum == 0.0f ? __int_as_float(0xff800000) : (top + (log2f(sum) - C::SHIFT)) * 0.6931471805599453f;
    }
}

// --------------------------------------------------------------------------------------- host

// n-tiles of eight rows: as few as hold a sequence's rows, at most what the registers hold.
int n_tiles(int64_t rows, int D) {
    if (rows <= 8) return 1;
    if (rows <= 16 || D == 256) return 2;
    return 4;
}

constexpr int kMaxCtasPerSm = 4;

template <int FMT, int D, int NT>
int run(const KvAttnArgs& a, cudaStream_t st) {
    using C = Cfg<FMT, D, NT>;
    auto kernel = kv_attention_kernel<FMT, D, NT>;
    auto join = kv_attention_join_kernel<FMT, D, NT>;
    // resident CTAs of an SM, asked once per device (0: not asked yet)
    static std::atomic<int> known[64];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ERR_CUDA;
    int per_sm = known[dev].load();
    if (per_sm == 0) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES) != cudaSuccess ||
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, kThreads, C::BYTES) != cudaSuccess || per_sm < 1)
            return MXQ_ERR_CUDA;
        if (per_sm > kMaxCtasPerSm) per_sm = kMaxCtasPerSm;
        known[dev].store(per_sm);
    }
    const int grid = sm_count() * per_sm;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = C::BYTES;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return MXQ_ERR_CUDA;
    cfg.gridDim = dim3(grid - 1, D / kJoinSlice);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join, a, grid) == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

template <int FMT>
int run_dim(int D, int nt, const KvAttnArgs& a, cudaStream_t st) {
    if (D == 64) return nt == 1 ? run<FMT, 64, 1>(a, st) : nt == 2 ? run<FMT, 64, 2>(a, st) : run<FMT, 64, 4>(a, st);
    if (D == 128) return nt == 1 ? run<FMT, 128, 1>(a, st) : nt == 2 ? run<FMT, 128, 2>(a, st) : run<FMT, 128, 4>(a, st);
    return nt == 1 ? run<FMT, 256, 1>(a, st) : run<FMT, 256, 2>(a, st);
}

}  // namespace

size_t kv_attention_workspace(int64_t batch, int64_t max_q, int heads, int kv_heads, int D) {
    (void)batch;
    const int rows = 8 * n_tiles(max_q * (heads / kv_heads), D);
    return static_cast<size_t>(sm_count()) * kMaxCtasPerSm * 2 * rows * (D + 2) * 4;
}

int launch_kv_attention(int fmt, int D, KvAttnArgs& a, cudaStream_t st) {
    const int nt = n_tiles(static_cast<int64_t>(a.max_q) * a.group, D);
    return fmt == MXQ_NVFP4 ? run_dim<MXQ_NVFP4>(D, nt, a, st) : run_dim<MXQ_MXFP4>(D, nt, a, st);
}

}  // namespace mxq
