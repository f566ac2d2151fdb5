// kv_attention.cu -- attention over the paged 4-bit key/value cache.
//
// One row tile is 8 NT rows (query token x query head of one kv head's group).  A warp turns a tile
// of cached tokens into matrix-instruction operands in registers and keeps its own running softmax:
//   S^T = K Q^T      m16n8k16, f16 x f16 -> fp32: tokens on M, rows on N, so that a group of up to
//                    eight rows wastes nothing and a decoded K operand serves all rows;
//   P   = 2^(c (s - m))  fp32, c > 0; m is the warp's running maximum of s, raised only when a tile exceeds it.  (The difference
//                    is taken before the factor: tokens of one score then weigh the same however large it is, and no
//                    exponent passes that of the maximum.)
//   O^T = V^T P^T    head channels on M, tokens on K.
// E2M1 codes convert to f16 exactly.  K: NVFP4 codes times their E4M3 scale are exact in f16 (six
// significant bits, at most 2688); MXFP4's power-of-two scale multiplies the fp32 product of its
// 32-element block.  Q is bf16 times a power of two per row (largest element in [2^7, 2^8)), exact in
// f16 but for elements 2^-24 below the row's largest.  V: the scale multiplies P instead of the codes,
// in f16: P is rounded to 11 bits (a bf16 P, 8 bits, would add as much error as the bf16 output has),
// times 2^7 (NVFP4) or 2^4 (MXFP4) so that small probabilities keep their bits.  MXFP4 scales are taken relative to a
// reference per 32 channels; a tile with scales that f16 does not hold beside it goes
// another way (wide_step), band by band of 12 codes, so that no value is lost beside another, seen or not.
// Sums, maxima and accumulators are fp32.
//
// Work is the list of all (sequence, row tile, kv head, token tile), cut evenly over the CTAs by every
// CTA for itself from the lengths on the device, so that ragged batches balance and a graph can be
// replayed with other lengths.  A CTA's part of a row tile that it does not have whole goes to the
// workspace as (m, l, O); a second kernel joins those in CTA order, so results do not depend on timing.
//
// What bounds it: beginning (5 us from the dependency to a CTA's first tile: lengths, page numbers and tiles, one
// round trip each), then about 5 TB/s of tiles (ALU pipe 50 % busy; the three CTAs of an SM come forward unequally,
// equal shares end up to 10 us apart), then the join (5 us).  40 heads, 8 kv heads of 128: one sequence of 131061 (NVFP4, 151 MB) 43.9 us, 32
// sequences of 500 to 16000 (MXFP4, 161 MB) 51.5 us, one of 1009 12.0 us; 24 heads, 4 kv heads of 256, a window
// of 2048 over 24 sequences of 90 to 9000 (MXFP4, 29 MB) 25.1 us.
#include <algorithm>
#include <atomic>

#include "kv_attn_common.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kWarps = 4;                     // warps that compute; one more feeds them
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kMinTiles = 4;     // token tiles a CTA gets at least (4, 8 and 12: 11.9, 12.9, 12.0 us for one sequence of 1009, MXFP4 12.1, 13.2, 12.5)
constexpr int kExtraTiles = 10;  // counted for beginning a row tile (32 sequences of 500 to 16000, MXFP4: 59.0 us at 0, 53.3 at 6, 51.5 at 10, 51.6 at 14)

template <int FMT, int D, int NT>
struct Cfg {
    using U = KvUnit<FMT, D>;
    static constexpr int TU = D <= 128 ? 2 : 1;  // units of a token tile
    static constexpr int TILE = 16 * TU;
    static constexpr int ROWS = 8 * NT;
    static constexpr int KS = D / 16;  // k steps of S, m tiles of O
    static constexpr int TILE_BYTES = TU * U::BYTES;
    static constexpr int OSTRIDE = D + 8;  // floats; row pairs of a warp's float2 stores meet different banks
    static constexpr int Q_BYTES = NT * KS * 32 * 8;
    static constexpr int RED = kWarps * ROWS * OSTRIDE * 4;
    // CTAs an SM holds, by registers (an accumulator of 4 NT KS a lane), and what is left of its shared memory
    static constexpr int CTAS = NT * KS <= 8 ? 3 : NT * KS <= 24 ? 2 : 1;
    static constexpr int BUDGET = (227 / CTAS - 1) * 1024 - 1024;
    static constexpr int FIXED = 2 * Q_BYTES + RED + 2 * (ROWS * 12 + 64) + kWarps * ROWS * 8 + 64;
    static constexpr int FIT = (BUDGET - FIXED) / (TILE_BYTES + 20);
    // A multiple of kWarps: tile n goes to warp n % kWarps, so that a slot's uses are all of one warp, in turn.
    // (Were they not, a warp could wait for use c of a slot whose use c - 1, another warp's, has not landed: the
    // barrier's one parity bit would let it pass.)
    static constexpr int STAGES = (FIT < 16 ? FIT : 16) / kWarps * kWarps;
    static_assert(STAGES >= 2 * kWarps, "shared memory");
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_Q = STAGES * TILE_BYTES;
    static constexpr int OFF_RED = OFF_Q + 2 * Q_BYTES;
    static constexpr int OFF_ROW = OFF_RED + RED;  // two buffers; per row: scale, first, end
    static constexpr int OFF_SEG = OFF_ROW + 2 * ROWS * 12;
    static constexpr int OFF_ML = OFF_SEG + 2 * 64;
    static constexpr int OFF_BAR = OFF_ML + kWarps * ROWS * 8;  // full, empty, segment full, segment empty
    static constexpr int OFF_SKIP = OFF_BAR + (2 * STAGES + 4) * 8;  // of each slot, a bit for each unit of a page outside the cache
    static constexpr int BYTES = OFF_SKIP + STAGES * 4;
    static_assert(sizeof(Segment) <= 64, "segment note");
    static constexpr float SHIFT = FMT == MXQ_NVFP4 ? 7.0f : 4.0f;  // log2 of what P is multiplied by
};

// --------------------------------------------------------------------------------- warp state

template <int FMT, int D, int NT>
struct Warp {
    using C = Cfg<FMT, D, NT>;
    float o[NT][C::KS][4];
    float base[NT][2], l[NT][2];  // probabilities are 2^(cs (s - base) + SHIFT): base is the running maximum of s
    // MXFP4, per 32 channels: E8M0 code that stands for 2^9 in the factors and in O.  It begins at 2^0, where most values'
    // scales are near, and follows a tile's largest code, within kRefMin and kRefMax, where that lies outside the band.  (O is
    // fp32 in units of 2^(ref - 136): it must not overflow beside values of 2^127, nor vanish beside a reference that
    // follows them up; so values of 2^-90 keep their bits beside any, and a reference above kRefDown stays.)
    int ref[FMT == MXQ_MXFP4 ? C::U::NB : 1];
    uint32_t bias;  // kBand - 3 - ref of the two blocks whose scales the lane checks, one a half
};
constexpr int kRefMin = 127 - 40, kRefMax = 127 + 40, kRefDown = 127 + 20;
// Scales that go into one product: codes ref - 9 to ref + 2, so factors 2^0 to 2^11.  P of 2^4 at most times the largest
// fits f16; below f16's normal range P is off by 2^-25 and its product by as much, together 2^-28 of the largest
// probability times the row's own largest value, whatever the reference follows.
constexpr int kBand = 12;

template <int FMT, int D, int NT>
__device__ __forceinline__ void warp_reset(Warp<FMT, D, NT>& w) {
    using C = Cfg<FMT, D, NT>;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < C::KS; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) w.o[n][j][i] = 0.0f;
        w.base[n][0] = w.base[n][1] = kNegMax;
        w.l[n][0] = w.l[n][1] = 0.0f;
    }
    if constexpr (FMT == MXQ_MXFP4) {
#pragma unroll
        for (int b = 0; b < C::U::NB; ++b) w.ref[b] = 127;
        w.bias = static_cast<uint32_t>((kBand - 3 - 127) & 0xFFFF) * 0x10001u;
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
                        float c[4];
                        mma_f16_first(c, lo[0], hi[0], lo[1], hi[1], q[n][0], q[n][1]);
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

// MXFP4, the V scales of a tile: a lane looks at four bytes, of a pair of tokens and two blocks (a dozen instructions a tile).
template <int D, int NT>
struct Scales {
    using C = Cfg<MXQ_MXFP4, D, NT>;
    using U = typename C::U;
    static constexpr int WORDS = C::TU * 4 * U::NB, PER = U::NB / 2;  // of the tile, of a pair of tokens
    static_assert(WORDS <= 32, "a word a lane");
    uint32_t x[1];

    __device__ __forceinline__ int word() const { return (threadIdx.x & 31) % WORDS; }
    __device__ __forceinline__ int which() const { return word() % PER; }  // blocks 2 which, 2 which + 1
    __device__ __forceinline__ void load(uint32_t tile) {
        lds<4>(tile + word() / (4 * U::NB) * U::BYTES + U::OFF_VS + 4 * (word() % (4 * U::NB)), x);
    }
    __device__ __forceinline__ void mask(int pos0, int seen0, int seen1, uint32_t skip) {  // what no row sees counts as zeros
        const int u = word() / (4 * U::NB);
        x[0] &= skip >> u & 1u ? 0u : pair_mask(pos0 + 16 * u + word() % (4 * U::NB) / PER * 2, seen0, seen1);
    }
    // either token's codes, a block a half, and code - ref + kBand - 3, in [0, kBand) if all is well (negative: a large unsigned one)
    __device__ __forceinline__ uint32_t codes(int token) const { return prmt(x[0], 0u, token ? 0x4341u : 0x4240u); }
    __device__ __forceinline__ uint32_t place(int token, const Warp<MXQ_MXFP4, D, NT>& w) const {
        return __viaddmax_s16x2(codes(token), w.bias, 0x80008000u);
    }
    __device__ __forceinline__ bool odd(const Warp<MXQ_MXFP4, D, NT>& w) const {
        const uint32_t most = __vmaxu2(place(0, w), place(1, w));
        // (a carry into the upper half comes from a lower one that is odd itself)
        return (((most + (0x8000u - kBand) * 0x10001u) | most) & 0x80008000u) != 0;
    }

    // Moves the references (and O) to the tile's largest scales where those lie outside the bands; whether scales remain
    // that do not go into one product.
    __device__ __forceinline__ bool refer(Warp<MXQ_MXFP4, D, NT>& w) const {
        uint32_t most = __vmaxu2(codes(0), codes(1));
#pragma unroll
        for (int o = PER; o < 32; o <<= 1) most = __vmaxu2(most, __shfl_xor_sync(0xffffffffu, most, o));
#pragma unroll
        for (int b = 0; b < U::NB; ++b) {
            const int code = __shfl_sync(0xffffffffu, most, b >> 1) >> (16 * (b & 1)) & 0xFFFF, to = min(max(code, kRefMin), kRefMax);
            if (code > w.ref[b] + 2 || (code != 0 && code < w.ref[b] + 3 - kBand && w.ref[b] <= kRefDown)) {
                const float f = __uint_as_float(static_cast<uint32_t>(w.ref[b] - to + 127) << 23);
                w.ref[b] = to;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 2 * b; j < 2 * b + 2; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) w.o[n][j][i] *= f;
            }
            const uint32_t half = static_cast<uint32_t>(kBand - 3 - w.ref[b]) & 0xFFFFu;
            if (which() == b >> 1) w.bias = b & 1 ? (w.bias & 0xFFFFu) | half << 16 : half;
        }
        // (code 0 counts as 0: the quantizer writes it for zeros, and for what is below 2^-124)
        uint32_t out = 0;
#pragma unroll
        for (int token = 0; token < 2; ++token) out |= codes(token) & ~__vcmpltu2(place(token, w), kBand * 0x10001u);
        return __any_sync(0xffffffffu, out != 0);
    }
};

// O += V^T P^T of one unit in bands of kBand codes: each product from zero, added to O in fp32 times the band's power of two.
template <int D, int NT>
__device__ __forceinline__ void wide_values(Warp<MXQ_MXFP4, D, NT>& w, const uint32_t (&p)[NT][2], const uint32_t (&sb)[2][D / 64],
                                            uint32_t unit) {
    using U = KvUnit<MXQ_MXFP4, D>;
    const int lane = threadIdx.x & 31;
#pragma unroll 1
    for (int band = (kRefMin + 2 - 255) / kBand - 1; band <= (kRefMax + 1) / kBand; ++band) {
        uint32_t fac[2][U::NB];
        bool some = false;
#pragma unroll
        for (int b = 0; b < U::NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                fac[h][b] = 0;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int code = sb[h][b >> 1] >> (16 * (b & 1) + 8 * half) & 0xFF, d = w.ref[b] + 2 - code - kBand * band;
                    if (code == 0 || d < 0 || d >= kBand) continue;
                    some = true;
                    fac[h][b] |= static_cast<uint32_t>(26 - d) << (10 + 16 * half);
                }
            }
        if (!__any_sync(0xffffffffu, some)) continue;
        static_assert(kBand % 2 == 0, "half of it as a factor, twice");
        const float f = __uint_as_float(static_cast<uint32_t>(127 - kBand / 2 * band) << 23);
#pragma unroll
        for (int wd = 0; wd < D / 64; ++wd) {
            uint32_t a[4][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {  // bytes 4 wd .. 4 wd + 3 of both tokens' D / 16 in this lane's record
                const int at0 = 4 * wd, at1 = D / 16 + 4 * wd;
                const uint32_t at = unit + U::OFF_V + h * (4 * D) + lane * U::W;
                uint32_t x[1], y[1];
                lds<4>(at + at0 / U::W * (32 * U::W) + at0 % U::W, x);
                lds<4>(at + at1 / U::W * (32 * U::W) + at1 % U::W, y);
                e2m1x8((x[0] & 0x0F0F0F0Fu) | (y[0] << 4 & 0xF0F0F0F0u), a[2 * h]);
                e2m1x8((x[0] >> 4 & 0x0F0F0F0Fu) | (y[0] & 0xF0F0F0F0u), a[2 * h + 1]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int j = 4 * wd + i;
                    float c[4];
                    mma_f16_first(c, a[0][i], a[1][i], a[2][i], a[3][i], hmul2(p[n][0], fac[0][j / 2]), hmul2(p[n][1], fac[1][j / 2]));
#pragma unroll
                    for (int k = 0; k < 4; ++k) w.o[n][j][k] = fmaf(c[k] * f, f, w.o[n][j][k]);
                }
        }
    }
}

// One token tile: scores, softmax update, O update.  pos0 is the tile's first token; MASK: some row does
// not see all of its tokens; seen0 / seen1: tokens that any row of the tile sees; skip: units that no row sees.  False for a
// tile of MXFP4 with V scales far apart, which has to be taken again with WIDE.  (Two
// copies of the code: with MASK for every tile 32 sequences take 75 to 84 us where they take 50 to 52.)
template <int FMT, int D, int NT, bool MASK, bool WIDE = false>
__device__ __forceinline__ bool tile_step(Warp<FMT, D, NT>& w, uint32_t tile, uint32_t qf, const float (&cs)[NT][2],
                                          const int* row_first, const int* row_end, int pos0, int seen0, int seen1, uint32_t skip) {
    using C = Cfg<FMT, D, NT>;
    using U = typename C::U;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    constexpr bool CHECK = FMT == MXQ_MXFP4 && !WIDE;
    Scales<D, NT> scales;
    if constexpr (CHECK) scales.load(tile);
    float s[C::TU][NT][4];
    scores<FMT, D, NT>(tile, qf, s);

    // one above SHIFT (all of them, before the first tile) raises the row's base
    auto masked = [&](int u, int n, int i, float v) {
        if constexpr (MASK) {
            const int pos = pos0 + 16 * u + 8 * (i >> 1) + g, r = 8 * n + 2 * t + (i & 1);
            if (pos < row_first[r] || pos >= row_end[r] || (skip >> u & 1u)) v = __int_as_float(0xff800000);
        }
        return v;
    };
    auto exponent = [&](int u, int n, int i, float base) {
        return masked(u, n, i, fmaf(s[u][n][i] - base, cs[n][i & 1], C::SHIFT));
    };
    float x[C::TU][NT][4];
    float top = kNegMax;
#pragma unroll
    for (int u = 0; u < C::TU; ++u)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[u][n][i] = exponent(u, n, i, w.base[n][i & 1]);
                top = fmaxf(top, x[u][n][i]);
            }
    bool odd = false;
    if constexpr (CHECK) {
        if constexpr (MASK) scales.mask(pos0, seen0, seen1, skip);
        odd = scales.odd(w);
    }
    if (__any_sync(0xffffffffu, top > C::SHIFT || odd)) {
        if constexpr (CHECK)
            if (__any_sync(0xffffffffu, odd) && scales.refer(w)) return false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float al[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float m = kNegMax;
#pragma unroll
                for (int u = 0; u < C::TU; ++u) m = fmaxf(m, fmaxf(masked(u, n, c, s[u][n][c]), masked(u, n, 2 + c, s[u][n][2 + c])));
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
                const float base = fmaxf(w.base[n][c], m);
                al[c] = ex2((w.base[n][c] - base) * cs[n][c]);
                w.base[n][c] = base;
                w.l[n][c] *= al[c];
#pragma unroll
                for (int u = 0; u < C::TU; ++u) {
                    x[u][n][c] = exponent(u, n, c, base);
                    x[u][n][2 + c] = exponent(u, n, 2 + c, base);
                }
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
            for (int i = 0; i < 4; ++i) e[i] = ex2(x[u][n][i]);
            w.l[n][0] += e[0] + e[2];
            w.l[n][1] += e[1] + e[3];
            p[n][0] = transpose8x8(cvt_f16x2(e[0], e[1]));
            p[n][1] = transpose8x8(cvt_f16x2(e[2], e[3]));
        }
        const uint32_t unit = tile + u * U::BYTES;
        // scale bytes of the pairs' tokens, then their factors, f16x2 per scale block
        constexpr int PB = 2 * U::NB;  // bytes of a token pair's scales
        uint32_t sb[2][PB / 4], fac[2][U::NB];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = unit + U::OFF_VS + (t + 4 * h) * PB;
            if constexpr (PB <= 16) {
                lds<PB>(at, sb[h]);
            } else {
                uint32_t y[4];
#pragma unroll
                for (int i = 0; i < PB / 16; ++i) {
                    lds<16>(at + 16 * i, y);
#pragma unroll
                    for (int k = 0; k < 4; ++k) sb[h][4 * i + k] = y[k];
                }
            }
        }
        if constexpr (MASK) {
            // P is 0 where a row does not see a token, but 0 times what is no number would not be: the scales
            // of tokens that no row sees become 0, and a NaN (the quantizer writes none) the largest number
            const int pos = pos0 + 16 * u + 2 * t;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t live = skip >> u & 1u ? 0u : pair_mask(pos + 8 * h, seen0, seen1);
#pragma unroll
                for (int i = 0; i < PB / 4; ++i) {
                    sb[h][i] &= live;
                    if constexpr (FMT == MXQ_NVFP4) sb[h][i] = __vminu4(sb[h][i] & 0x7F7F7F7Fu, 0x7E7E7E7Eu);
                }
            }
        }
        if constexpr (WIDE) {
            wide_values<D, NT>(w, p, sb, unit);
            continue;
        }
        if constexpr (FMT == MXQ_NVFP4) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int b = 0; b < U::NB; ++b) fac[h][b] = e4m3x2_f16x2(b & 1 ? sb[h][b >> 1] >> 16 : sb[h][b >> 1] & 0xFFFFu);
        } else {
            // 2^(code - ref + 9): the exponent fields code - ref + 24 of both halves; 0 for code 0, as any ref is above 24
#pragma unroll
            for (int b = 0; b < U::NB; ++b) {
                const uint32_t bias = static_cast<uint32_t>((24 - w.ref[b]) & 0xFFFF) * 0x10001u;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t codes = prmt(sb[h][b >> 1], 0u, b & 1 ? 0x4342u : 0x4140u);  // one a half
                    fac[h][b] = __viaddmax_s16x2_relu(codes, bias, 0u) << 10;
                }
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
                    mma_f16(w.o[n][j], a[0][i], a[1][i], a[2][i], a[3][i], b0, b1);
                }
            }
        }
    }
    return true;
}

// The same for token tile i of a segment of MXFP4, with scales far apart.  Rare, and out of line.
template <int D, int NT>
__device__ __noinline__ void wide_copy(Warp<MXQ_MXFP4, D, NT>& w, const uint8_t* smem, uint32_t buf, int i) {
    using C = Cfg<MXQ_MXFP4, D, NT>;
    const Segment& seg = *reinterpret_cast<const Segment*>(smem + C::OFF_SEG + buf * 64);
    const float* row_scale = reinterpret_cast<const float*>(smem + C::OFF_ROW + buf * C::ROWS * 12);
    const int* row_first = reinterpret_cast<const int*>(row_scale + C::ROWS);
    const uint32_t slot = (seg.base + i) % C::STAGES;
    float cs[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) cs[n][c] = row_scale[8 * n + 2 * (threadIdx.x & 3) + c];
    tile_step<MXQ_MXFP4, D, NT, true, true>(w, smem_u32(smem + C::OFF_RING + slot * C::TILE_BYTES),
                                            smem_u32(smem + C::OFF_Q + buf * C::Q_BYTES), cs, row_first, row_first + C::ROWS,
                                            seg.pos0 + i * C::TILE, seg.seen0, seg.seen1,
                                            reinterpret_cast<const volatile uint32_t*>(smem + C::OFF_SKIP)[slot]);
}
template <int D, int NT>
__device__ __forceinline__ void wide_step(Warp<MXQ_MXFP4, D, NT>& w, const uint8_t* smem, uint32_t buf, int i) {
    Warp<MXQ_MXFP4, D, NT> copy = w;  // (so that the state itself stays in registers)
    wide_copy<D, NT>(copy, smem, buf, i);
    w = copy;
}

// ------------------------------------------------------------------------------------- kernel

// The feeding warp: walks the CTA's work, notes each segment and its Q operands (two buffers), and keeps
// the ring of token tiles full, so that the computing warps never wait for an index or a query.
template <int FMT, int D, int NT>
__device__ __forceinline__ void feed(const KvAttnArgs& a, uint8_t* smem) {
    using C = Cfg<FMT, D, NT>;
    using U = typename C::U;
    const int lane = threadIdx.x & 31;
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + C::STAGES;
    uint64_t* seg_full = empty + C::STAGES;
    uint64_t* seg_empty = seg_full + 2;

    const Plan plan = make_plan<C::TILE, C::ROWS, kExtraTiles>(a, kMinTiles);
    if (lane == 0) reinterpret_cast<Split*>(a.partial)[blockIdx.x].parts = 0;
    int64_t at = plan.at, off = plan.off;
    const int64_t stop = min(at + plan.per, plan.work);
    int b = plan.b, qt = plan.qt;
    Seq s = plan.s;
    float qscale = a.scale * 1.4426950408889634f;
    if constexpr (FMT == MXQ_NVFP4) qscale *= *a.g_k;
    const uint32_t flip = qscale < 0.0f ? 0x80008000u : 0u;  // Q takes the sign
    qscale = fabsf(qscale);
    uint32_t tiles = 0, nseg = 0;

#pragma unroll 1
    for (;; ++nseg) {
        const uint32_t buf = nseg & 1u;
        Segment* note = reinterpret_cast<Segment*>(smem + C::OFF_SEG + buf * 64);
        // the row tile and kv head that hold work item `at`: its token tiles [from, from + count) of n
        int t0 = 0, n = 0, head = 0, from = 0, count = 0;
        int64_t place = 0, share = 0;  // of the work counted for it
#pragma unroll 1
        while (at < stop) {
            if (qt * C::ROWS >= s.qn * a.group) {
                s = load_seq(a, ++b);
                qt = 0;
                continue;
            }
            const TileSpan span = tile_span<C::TILE, C::ROWS>(a, s.kv, s.qn, qt);
            t0 = span.first, n = span.count;
            const int64_t each = n + kExtraTiles;  // of a head
            if (off >= each * a.kv_heads) {
                off -= each * a.kv_heads;
                ++qt;
                continue;
            }
            head = div_small(off, each, place);
            share = min(each - place, stop - at);
            from = max(static_cast<int>(place) - kExtraTiles, 0);
            count = max(static_cast<int>(place + share) - kExtraTiles, 0) - from;
            if (count > 0) break;
            at += share;  // nothing but tiles that are only counted
            off += share;
        }
        if (count == 0) {
            if (!wait_warp(&seg_empty[buf], (nseg >> 1 & 1u) ^ 1u, a.status, 0x41)) return;
            if (lane == 0) {
                note->count = -1;
                mbar_arrive(&seg_full[buf]);
            }
            return;
        }
        const int row0 = qt * C::ROWS, rows = min(C::ROWS, s.qn * a.group - row0);
        int seen0, seen1, all0, all1;
        row_span(a, s, row0, seen0, all1);
        row_span(a, s, row0 + rows - 1, all0, seen1);

        // A lane has every BATCH-th token tile: it finds the tile's units (byte offsets, -1: not loaded) one
        // batch ahead and starts the copies itself when their ring slot is free.  (One elected lane that did all
        // of it took 600 cycles a tile, three times what HBM takes to deliver one.)
        constexpr int BATCH = 8;
        static_assert(BATCH <= C::STAGES, "a slot comes up once in a batch: its barrier has one parity bit");
        const int first_unit = (t0 + from) * C::TU;
        // In front of and behind the tokens that some row sees, pages may not exist (a window's may have been given away)
        const int units_from = seen0 >> 4, units_end = min((seen1 + 15) >> 4, first_unit + count * C::TU);
        int page[C::TU], in_page[C::TU];  // of the lane's units of the next batch; page is not looked at before it is used
        auto look_up = [&](int tile) {    // for the batch that begins at `tile`
#pragma unroll
            for (int u = 0; u < C::TU; ++u) {
                const int unit = first_unit + (tile + lane) * C::TU + u;
                const int at_page = a.page_units == 1 ? unit : static_cast<int>(__umulhi(unit, a.page_magic));  // unit / page_units
                in_page[u] = lane < BATCH && unit >= units_from && unit < units_end ? unit - at_page * a.page_units : -1;
                page[u] = 0;
                if (in_page[u] >= 0) page[u] = a.table[static_cast<int64_t>(b) * a.table_stride + at_page];
            }
        };
        look_up(0);
        // Q rows in flight beside them: lane (g, t) takes what it needs of row g as the B operand of S, 8
        // elements (two k steps) a load, as the K codes are dealt to the lanes
        constexpr int LOADS = D / 32;
        const int g = lane >> 2, t = lane & 3;
        uint4 x[LOADS];
        auto load_rows = [&](int r8) {
            const int row = row0 + r8 + g, j = a.max_q == 1 ? 0 : row / a.group;
            const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<int64_t>(s.q0 + j) * a.q_token_stride +
                                                              static_cast<int64_t>(head * a.group + row - j * a.group) * a.q_head_stride);
#pragma unroll
            for (int i = 0; i < LOADS; ++i) {
                x[i] = make_uint4(0, 0, 0, 0);
                if (r8 + g < rows) x[i] = src[FMT == MXQ_NVFP4 ? t * LOADS + i : i * 4 + t];
            }
        };
        load_rows(0);
        if (!wait_warp(&seg_empty[buf], (nseg >> 1 & 1u) ^ 1u, a.status, 0x41)) return;
        if (lane == 0) {
            note->count = count;
            note->base = tiles;
            note->pos0 = (t0 + from) * C::TILE;
            note->seen0 = seen0, note->seen1 = seen1, note->all0 = all0, note->all1 = all1;
            note->q0 = s.q0, note->row0 = row0, note->rows = rows, note->head = head;
            note->begins = from == 0;
            note->whole = from == 0 && count == n;
            int64_t rest;
            note->parts = from == 0 ? div_small(at - place + kExtraTiles + n - 1, plan.per, rest) - static_cast<int>(blockIdx.x) + 1 : 0;
        }
        // The first segment's copies start in front of its note (the ring is empty); later ones behind it,
        // as their slots come free only while the computing warps are at the segment before.
        int issued = 0, limit = nseg == 0 ? min(count, C::STAGES / BATCH * BATCH) : 0;
#pragma unroll 1
        for (int phase = 0; phase < 2; ++phase, limit = count) {
#pragma unroll 1
            for (; issued < limit; issued += BATCH) {
                int64_t src[C::TU];
                uint32_t skip = 0;
#pragma unroll
                for (int u = 0; u < C::TU; ++u) {
                    src[u] = -1;
                    if (in_page[u] < 0) continue;
                    if (page[u] < 0 || page[u] >= a.num_pages) {
                        kv_status(a.status, kStatusKvPage);
                        skip |= 1u << u;
                        continue;
                    }
                    src[u] = (static_cast<int64_t>(page[u]) * a.kv_heads + head) * a.page_bytes +
                             static_cast<int64_t>(in_page[u]) * U::BYTES;
                }
                look_up(issued + BATCH);
                const uint32_t n = tiles + issued + lane, slot = n % C::STAGES, parity = (n / C::STAGES & 1u) ^ 1u;
                bool todo = lane < BATCH && issued + lane < count;
                uint64_t since = 0;
#pragma unroll 1
                for (uint32_t polls = 0; __any_sync(0xffffffffu, todo); ++polls) {
                    if (todo && mbar_test_wait(&empty[slot], parity)) {
                        todo = false;
                        uint8_t* dst = smem + C::OFF_RING + slot * C::TILE_BYTES;
                        reinterpret_cast<uint32_t*>(smem + C::OFF_SKIP)[slot] = skip;  // (in front of the arrival below)
                        uint32_t bytes = 0;
#pragma unroll
                        for (int u = 0; u < C::TU; ++u) bytes += src[u] < 0 ? 0 : U::BYTES;
                        mbar_arrive_expect_tx(&full[slot], bytes);
                        if (C::TU == 2 && src[0] >= 0 && src[C::TU - 1] == src[0] + U::BYTES) {  // neighbours in one page
                            bulk_load(dst, a.cache + src[0], 2 * U::BYTES, &full[slot]);
                        } else {
#pragma unroll
                            for (int u = 0; u < C::TU; ++u)
                                if (src[u] >= 0) bulk_load(dst + u * U::BYTES, a.cache + src[u], U::BYTES, &full[slot]);
                        }
                    }
                    __syncwarp();
                    if ((polls & 255u) == 255u) {  // (a bounded wait, as all others)
                        if (since == 0) since = globaltimer();
                        if (__any_sync(0xffffffffu, globaltimer() - since > kWaitLimitNs)) {
                            if (lane == 0) atomicCAS(a.status, 0, kStatusTimeoutBase + 0x42);
                            return;
                        }
                    }
                }
            }
            if (phase == 1) break;
            // Q operands: rows as f16 times a power of two
            float* row_scale = reinterpret_cast<float*>(smem + C::OFF_ROW + buf * C::ROWS * 12);
            int* row_first = reinterpret_cast<int*>(row_scale + C::ROWS);
            int* row_end = row_first + C::ROWS;
#pragma unroll 1
            for (int r8 = 0; r8 < C::ROWS; r8 += 8) {
                if (r8) load_rows(r8);
                uint32_t top = 0;  // bf16 magnitudes order like integers
#pragma unroll
                for (int i = 0; i < LOADS; ++i)
                    top = __vmaxu2(__vmaxu2(top, __vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu)),
                                   __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
                uint32_t big = max(top & 0xFFFFu, top >> 16);
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = max(big, __shfl_xor_sync(0xffffffffu, big, 2));
                const uint32_t ex = max(big >> 7, 8u);
                const float mul = __uint_as_float((261u - ex) << 23);
                uint8_t* dst = smem + C::OFF_Q + buf * C::Q_BYTES + (r8 / 8) * (C::KS / 2) * 512 + lane * 16;
#pragma unroll
                for (int i = 0; i < LOADS; ++i) {
                    const uint32_t y[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t h[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        h[k] = cvt_f16x2(__uint_as_float(y[k] << 16) * mul, __uint_as_float(y[k] & 0xFFFF0000u) * mul) ^ flip;
                    *reinterpret_cast<uint4*>(dst + i * 512) = make_uint4(h[0], h[1], h[2], h[3]);
                }
                if (t == 0) {
                    const int r = r8 + g;
                    row_scale[r] = qscale * __uint_as_float((ex - 7u) << 23);
                    int f0 = 0, f1 = 0;
                    if (r < rows) row_span(a, s, row0 + r, f0, f1);
                    row_first[r] = f0;
                    row_end[r] = f1;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&seg_full[buf]);
        }
        tiles += count;
        at += share;
        off += share;
    }
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<FMT, D, NT>::CTAS) kv_attention_kernel(const __grid_constant__ KvAttnArgs a) {
    using C = Cfg<FMT, D, NT>;
    extern __shared__ __align__(128) uint8_t smem[];
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
    uint64_t* empty = full + C::STAGES;
    uint64_t* seg_full = empty + C::STAGES;
    uint64_t* seg_empty = seg_full + 2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = lane & 3, g = lane >> 2;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], kWarps);
        }
        fence_barrier_init();
    }
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait();
    if (warp == kWarps) {
        feed<FMT, D, NT>(a, smem);
        return;
    }

    float* partials = a.partial + gridDim.x * (sizeof(Split) / 4);
    float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    bool dead = false;
#pragma unroll 1
    for (uint32_t nseg = 0;; ++nseg) {
        const uint32_t buf = nseg & 1u;
        dead = !wait_warp(&seg_full[buf], nseg >> 1 & 1u, a.status, 0x43);
        // one decision for the computing warps; also: the last segment's O has been read
        if (named_barrier_or(1, kWarps * 32, dead)) return;
        const Segment& seg = *reinterpret_cast<const Segment*>(smem + C::OFF_SEG + buf * 64);
        const int count = seg.count;
        if (count < 0) return;
        const float* row_scale = reinterpret_cast<const float*>(smem + C::OFF_ROW + buf * C::ROWS * 12);
        const int* row_first = reinterpret_cast<const int*>(row_scale + C::ROWS);
        const int* row_end = row_first + C::ROWS;
        const uint32_t qf = smem_u32(smem + C::OFF_Q + buf * C::Q_BYTES);
        const int seen0 = seg.seen0, seen1 = seg.seen1, all0 = seg.all0, all1 = seg.all1;
        const uint32_t base = seg.base;
        float cs[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) cs[i][c] = row_scale[8 * i + 2 * t + c];

        Warp<FMT, D, NT> w;
        warp_reset(w);
        // tile i of the segment is tile base + i of the CTA, which warp (base + i) % kWarps takes
        int first = warp - static_cast<int>(base % kWarps);
        if (first < 0) first += kWarps;
        int pos0 = seg.pos0 + first * C::TILE;
        int i = first;
#pragma unroll 1
        for (;;) {
            bool done = true;
#pragma unroll 1
            for (; i < count; i += kWarps, pos0 += kWarps * C::TILE) {
                const uint32_t slot = (base + i) % C::STAGES;
                if (!wait_warp(&full[slot], (base + i) / C::STAGES & 1u, a.status, 0x40)) {
                    dead = true;
                    break;
                }
                const uint32_t tile = smem_u32(smem + C::OFF_RING + slot * C::TILE_BYTES);
                const uint32_t skip = reinterpret_cast<const volatile uint32_t*>(smem + C::OFF_SKIP)[slot];
                done = skip == 0 && pos0 >= all0 && pos0 + C::TILE <= all1
                           ? tile_step<FMT, D, NT, false>(w, tile, qf, cs, row_first, row_end, pos0, seen0, seen1, 0)
                           : tile_step<FMT, D, NT, true>(w, tile, qf, cs, row_first, row_end, pos0, seen0, seen1, skip);
                if (!done) break;
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[slot]);
            }
            if (FMT == MXQ_NVFP4 || done) break;
            if constexpr (FMT == MXQ_MXFP4) {
                // (All that this needs is found again from the note: what the loop above kept for it in registers, it paid
                // for in spills, 3 % of its time.)
                int k = i;
                asm volatile("" : "+r"(k));
                wide_step<D, NT>(w, smem, buf, k);
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[(seg.base + k) % C::STAGES]);
                i = k + kWarps, pos0 = seg.pos0 + i * C::TILE;
            }
        }

        // join the warps: each leaves (base in units of log 2, l, O); the sums are taken by all together
#pragma unroll
        for (int i = 0; i < NT; ++i) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float x = w.l[i][c];
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                // (x is 0 where the warp has seen no token, and at least 2^SHIFT else)
                if (g == 0)
                    ml[warp * C::ROWS + 8 * i + 2 * t + c] = make_float2(x == 0.0f ? kNegMax : w.base[i][c] * cs[i][c] - C::SHIFT, x);
            }
#pragma unroll
            for (int j = 0; j < C::KS; ++j) {
                float x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k] = w.o[i][j][k];
                    if constexpr (FMT == MXQ_MXFP4) x[k] = scale_pow2(x[k], w.ref[j / 2] - 136);
                }
                float* dst = red + (warp * C::ROWS + 8 * i + 2 * t) * C::OSTRIDE + 16 * j + 2 * g;
                *reinterpret_cast<float2*>(dst) = make_float2(x[0], x[2]);
                *reinterpret_cast<float2*>(dst + C::OSTRIDE) = make_float2(x[1], x[3]);
            }
        }
        if (named_barrier_or(1, kWarps * 32, dead)) return;
        const int q0 = seg.q0, row0 = seg.row0, rows = seg.rows, head = seg.head;
        const bool whole = seg.whole, begins = seg.begins;
        // parts: a CTA has at most one that begins its row tile (the second slot) and one that does not
        float* part = partials + (static_cast<int64_t>(blockIdx.x) * 2 + (begins ? 1 : 0)) * (C::ROWS * (D + 2));
        if (begins && !whole && threadIdx.x == 0) {
            Split* split = reinterpret_cast<Split*>(a.partial) + blockIdx.x;
            split->parts = seg.parts;
            split->q0 = q0;
            split->row0 = row0;
            split->rows = rows;
            split->head = head;
        }
        float gv = 1.0f;
        if (FMT == MXQ_NVFP4 && whole) gv = *a.g_v;
#pragma unroll 1
        for (int i = threadIdx.x; i < C::ROWS * (D / 4); i += kWarps * 32) {
            const int r = i / (D / 4), d = i % (D / 4) * 4;
            float top = kNegMax, sum = 0.0f;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) top = fmaxf(top, ml[k * C::ROWS + r].x);
#pragma unroll
            for (int k = 0; k < kWarps; ++k) {
                const float2 z = ml[k * C::ROWS + r];
                const float f = ex2(z.x - top);
                const float4 v = *reinterpret_cast<const float4*>(red + (k * C::ROWS + r) * C::OSTRIDE + d);
                sum = fmaf(z.y, f, sum);
                x.x = fmaf(v.x, f, x.x);
                x.y = fmaf(v.y, f, x.y);
                x.z = fmaf(v.z, f, x.z);
                x.w = fmaf(v.w, f, x.w);
            }
            if (whole) {
                if (r < rows) {
                    const int row = row0 + r, j = a.max_q == 1 ? 0 : row / a.group;
                    const int64_t o = static_cast<int64_t>(q0 + j) * a.heads + head * a.group + row - j * a.group;
                    const float inv = gv * (sum > 0.0f ? 1.0f / sum : sum);  // sum is 0 (no token) or not a number
                    put4(a, o * D + d, x.x * inv, x.y * inv, x.z * inv, x.w * inv);
                    if (a.lse && d == 0)
                        a.lse[o] = sum == 0.0f ? __int_as_float(0xff800000) : (top + log2f(sum)) * 0.6931471805599453f;
                }
            } else {
                *reinterpret_cast<float4*>(part + r * D + d) = x;
                if (d == 0) *reinterpret_cast<float2*>(part + C::ROWS * D + 2 * r) = make_float2(top, sum);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&seg_empty[buf]);
    }
}

// --------------------------------------------------------------------------------------- host

// n-tiles of eight rows a CTA takes at once, one or two: the second one costs 3/4 of the first (head size 256: 8/9), as
// K and V are decoded already, but the last row tile pads to 16 rows.  16 sequences of 3000 to 4100, with one and
// with two, in us: head size 128, MXFP4, 10 rows 42 and 37, 20 rows 56 and 58, 35 rows 83 and 80; 64, 10 rows 31 and 28,
// 35 rows 57 and 52; head size 256, 10 rows 71 and 69, 20 rows 99 and 124, 50 rows 210 and 228, 500 rows 1745 and 1685.
// Three or four leave room for half the warps (slower by 6 to 11 % for a chunk of 700 tokens).
int n_tiles(int64_t rows, int D) {
    const int64_t ones = (rows + 7) / 8, twos = 2 * ((rows + 15) / 16);
    return (D == 256 ? 9 * ones < 8 * twos : ones == 1) ? 1 : 2;
}

// Rows from which a row tile on tcgen05 (32 rows for NVFP4 with head size 128, else 128) takes less time.  16
// sequences of 3000 to 4100, 8 kv heads, here and there, in us: NVFP4, 128 wide, 10 rows 35 and 47, 20 rows 55 and
// 48, 35 rows 76 and 71, 65 rows 117 and 73; 64 wide, 35 rows 51 and 58, 50 rows 63 and 59, 65 rows 75 and 59; MXFP4, 128
// wide, 35 rows 80 and 85, 50 rows 102 and 86, 65 rows 123 and 87, 500 rows 689 and 254; 64 wide, 35 rows 51 and 66, 50
// rows 64 and 67, 65 rows 76 and 67, 500 rows 397 and 201.
bool on_tcgen05(int fmt, int D, int64_t rows) {
    return D <= 128 && rows > (fmt == MXQ_NVFP4 && D == 128 ? 16 : 48);
}

constexpr int kMaxCtasPerSm = 4;

template <int FMT, int D, int NT>
int run(KvAttnArgs& a, cudaStream_t st) {
    using C = Cfg<FMT, D, NT>;
    auto kernel = kv_attention_kernel<FMT, D, NT>;
    auto join = kv_attention_join_kernel<FMT, D, C::ROWS>;
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
    const int grid = std::min(sm_count() * per_sm, kMaxGrid);
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
    a.inv_grid = 1.0f / static_cast<float>(grid);
    if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return MXQ_ERR_CUDA;
    cfg.gridDim = dim3(2 * sm_count());
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, join, a, grid) == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

template <int FMT>
int run_dim(int D, int nt, KvAttnArgs& a, cudaStream_t st) {
    if (D == 64) return nt == 1 ? run<FMT, 64, 1>(a, st) : run<FMT, 64, 2>(a, st);
    if (D == 128) return nt == 1 ? run<FMT, 128, 1>(a, st) : run<FMT, 128, 2>(a, st);
    return nt == 1 ? run<FMT, 256, 1>(a, st) : run<FMT, 256, 2>(a, st);
}

}  // namespace

size_t kv_attention_workspace(int64_t batch, int64_t max_q, int heads, int kv_heads, int D) {
    (void)batch;
    const int64_t rows = max_q * (heads / kv_heads);
    const size_t here = static_cast<size_t>(sm_count()) * kMaxCtasPerSm * (2 * 8 * n_tiles(rows, D) * (D + 2) * 4 + sizeof(Split));
    const size_t there = static_cast<size_t>(sm_count()) * (2 * kv_rows_tile(rows) * (D + 2) * 4 + sizeof(Split));
    return rows > 16 && D <= 128 ? std::max(here, there) : here;
}

int launch_kv_attention(int fmt, int D, KvAttnArgs& a, cudaStream_t st) {
    const int64_t rows = static_cast<int64_t>(a.max_q) * a.group;
    if (on_tcgen05(fmt, D, rows)) return launch_kv_attention_rows(fmt, D, a, st);
    const int nt = n_tiles(rows, D);
    return fmt == MXQ_NVFP4 ? run_dim<MXQ_NVFP4>(D, nt, a, st) : run_dim<MXQ_MXFP4>(D, nt, a, st);
}

}  // namespace mxq
