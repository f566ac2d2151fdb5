// kv_attention_rows.cu -- attention over the paged 4-bit cache for sequences with many rows (query token x
// query head of a kv head's group): drafted tokens, chunks of a prefill.  on_tcgen05 in kv_attention.cu says
// from how many rows on.
//
// With many rows the tensor work counts, so it runs on tcgen05 (kind::f16, fp32 accumulators in TMEM), one
// CTA per SM, tiles of 128 tokens:
//   S = Q K^T   Q [128 rows x D] and K in shared memory, 128-byte swizzle; Q once per segment, times a power of two per
//               row; K codes times scale;
//   P = 2^(s - base) in TMEM; one thread has one row, so the softmax needs no shuffles;
//   O += P V    V codes times scale in shared memory, transposed ([channel][token]).
// NVFP4 operands are f16, which holds codes times E4M3 scales exactly, and P rounded to 11 bits.  MXFP4 operands are bf16:
// codes times E8M0 scales need two bits and the whole range of exponents, which f16 does not have.  (As f16 relative to a
// running reference, blocks 2^23 below it vanished, and eight warps agreed on that reference in every tile: 5 % slower.)
// P is two bf16 then, its upper and its lower 8 bits, and O two products.
// Roles: two groups of 4 softmax warps (their TMEM lanes are the rows) that take the tiles in turn, each with
// its own S and O, so that one group's exponentials run beside the other's products; 4 warps that decode K
// (32 tokens of a tile each) and 8 that decode V (16 tokens); one warp that feeds raw tiles by bulk copies;
// one that issues the MMAs.  P takes the place of S, of its first half as f16: chunk by chunk of 32 tokens the scores are
// read, and their probabilities written where scores have been read already.
// QUAD (up to 32 rows): the rows stand four times in the lanes, and each softmax warp takes 32 of the tile's 128
// tokens, the others' P columns being zero: the four partial results join at the end, like CTAs' parts.  NVFP4 with heads
// of 128 alone: 20 rows of MXFP4 took 80 us so and 55 in kv_attention.cu, and heads of 64 take 38 there.
// The base of a row follows its maximum only when a probability would pass 2^15 (f16 ends at 2^16); O and
// the tile's earlier P are rescaled in TMEM then.  Work is cut over the CTAs as in kv_attention.cu, with the
// same join kernel.
//
// What bounds it (NVFP4): a tile takes 2200 to 2500 cycles.  The products alone take 1750: eight instructions of S and of
// P V are issued in 870 cycles each, not the 512 of an idle SM, as K, V and Q are read from shared memory beside the
// decoders' writes (about 200 KB a tile at 128 bytes a cycle).  A softmax group of 128 rows needs 3600 cycles for
// 128 scores a thread, two groups in turn.  Beside that a segment ends in 5000 to 10000 cycles (the last product,
// joining the groups); with Q brought by the softmax warps afterwards, not by the value warps meanwhile, a chunk took
// 11 us more.  Giving raw tiles back before the wait for the operand's place changed nothing.
// A chunk of 700 tokens over 2 sequences of 4200 to 8300 (40 heads, 8 kv heads of 128): 194 us for NVFP4
// (583 TFLOP/s), 242 for MXFP4, whose P V is two products.  Four drafted tokens for each of 16 sequences of 3000 to
// 4100 (NVFP4): 49 us.
#include <algorithm>
#include <atomic>

#include "kv_attn_common.cuh"
#include "mxq_internal.h"

namespace mxq {
namespace {

constexpr int kSoftWarps = 8, kKeyWarps = 4, kValueWarps = 8, kDecWarps = kKeyWarps + kValueWarps;
static_assert(kSoftWarps == 8 && kValueWarps == 8, "either bring Q");
constexpr int kFeedWarp = kSoftWarps + kDecWarps, kMmaWarp = kFeedWarp + 1;
constexpr int kRowThreads = (kMmaWarp + 1) * 32;
constexpr int kTokens = 128;  // of a tile
constexpr int kMinRowTiles = 2;
constexpr float kStart = 7.0f, kLimit = 15.0f;  // a fresh base puts the maximum at 2^6 to 2^7; above 2^15 it is raised

template <int FMT, int D, bool QUAD>
struct RCfg {
    using U = KvUnit<FMT, D>;
    static constexpr int ROWS = QUAD ? 32 : 128;
    // Tiles counted for beginning a row tile: a chunk of 700 takes 195 us at 3 and 5, 201 at 8, 208 at 12 (MXFP4 239,
    // 242, 250, 259); four drafted tokens 49.6 at 5, 49.5 at 8, 49.0 at 12, 50.0 at 16.
    static constexpr int EXTRA = QUAD ? 12 : 5;
    static constexpr int UNITS = kTokens / 16;
    static constexpr int RAW = UNITS * U::BYTES;
    static constexpr int STAGES = 3;
    static constexpr int K16 = kTokens * D * 2, V16 = kTokens * D * 2, Q16 = 128 * D * 2;  // bytes of an operand
    static constexpr int OFF_K = 0;  // 1024-byte aligned, as the others
    static constexpr int OFF_V = OFF_K + 2 * K16;
    static constexpr int OFF_Q = OFF_V + 2 * V16;  // QUAD: at a segment's end also [4][32][MERGE] floats
    static constexpr int MERGE = 33;               // floats: a slice of 32 channels and a skew
    static_assert(!QUAD || (FMT == MXQ_NVFP4 && D == 128 && 4 * 32 * MERGE * 4 <= Q16), "what is joined in one CTA");
    static constexpr int OFF_RAW = OFF_Q + Q16;
    static constexpr int OFF_ML = OFF_RAW + STAGES * RAW;  // [2 groups][128 lanes] (base, l)
    static constexpr int OFF_QS = OFF_ML + 2 * 128 * 8;  // scale of each row's scores, two buffers
    // of the last eight tiles, a bit for each unit of a page outside the cache (a tile is eight behind only when its
    // softmax is done: it is decoded before the third tile behind it is fed, the second's V waits for its product)
    static constexpr int OFF_SKIP = OFF_QS + 2 * 128 * 4;
    static constexpr int OFF_SEG = OFF_SKIP + 8 * 4;
    static constexpr int OFF_BAR = OFF_SEG + 2 * 64;
    static constexpr int NBARS = 2 * STAGES + 10 + 1 + 4;
    static constexpr int OFF_TMEM = OFF_BAR + NBARS * 8;
    static constexpr int BYTES = OFF_TMEM + 16 + 1024;  // and the alignment
    static constexpr uint32_t S_COL = 0, O_COL = 256;   // two of each: S 128 columns, O D columns
};

struct RowBars {
    uint64_t *raw_full, *raw_empty, *kf, *vf, *sf, *pf, *od, *qf, *seg_full, *seg_empty;
    __device__ __forceinline__ RowBars(uint8_t* at, int stages) {
        uint64_t* b = reinterpret_cast<uint64_t*>(at);
        raw_full = b, raw_empty = b + stages, b += 2 * stages;
        // of tile n, at n & 1: K and V decoded, S done (K may be overwritten), P written, O done (V, P may be)
        kf = b, vf = b + 2, sf = b + 4, pf = b + 6, od = b + 8, b += 10;
        qf = b, b += 1;
        seg_full = b, seg_empty = b + 2;
    }
};

// Units of tile n that no row sees, as the feeding warp noted them.
template <class C>
__device__ __forceinline__ uint32_t skipped(const uint8_t* smem, uint32_t n) {
    return reinterpret_cast<const volatile uint32_t*>(smem + C::OFF_SKIP)[n & 7];
}

// MXFP4 operands are codes times 2^(scale code - 127 - offset): scale codes up to 255 stay finite with what E2M1 adds, and
// sums of products with P (2^15 at most) or Q (2^8) within fp32 for values up to 2^113 and more.
constexpr int kKeyOffset = 12, kValueOffset = 20;

// 8 E2M1 codes as 4 bf16x2, times 2^-126: byte i of w becomes o[i], its low nibble in the low half (see dequant8_mul).
__device__ __forceinline__ void e2m1x8_tiny(uint32_t w, uint32_t (&o)[4]) {
    const uint32_t ev = w & 0x0F0F0F0Fu, od = w >> 4 & 0x0F0F0F0Fu;
    o[0] = prmt(ev, od, 0x8480u) * 0x1040u & 0x81C081C0u;
    o[1] = prmt(ev, od, 0x9591u) * 0x1040u & 0x81C081C0u;
    o[2] = prmt(ev, od, 0xA6A2u) * 0x1040u & 0x81C081C0u;
    o[3] = prmt(ev, od, 0xB7B3u) * 0x1040u & 0x81C081C0u;
}
__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Scale codes c, one a half: bf16x2 factors for e2m1x8_tiny, 2^(126 + c - 127 - offset) as far as bf16 goes, and what is
// left of codes behind that.
template <int OFFSET>
struct MxFactor {
    static constexpr uint32_t LAST = 128 + OFFSET;  // 2^127
    uint32_t first, rest;
    bool more;
    __device__ __forceinline__ explicit MxFactor(uint32_t c) {
        const uint32_t low = __vminu2(c, LAST * 0x10001u);
        first = (low + (126u - OFFSET) * 0x10001u) << 7;
        rest = (c - low + 127u * 0x10001u) << 7;
        more = c != low;
    }
    __device__ __forceinline__ uint32_t of(uint32_t x) const {
        x = bmul2(x, first);
        return more ? bmul2(x, rest) : x;
    }
};

// Feeds raw tiles (whole warp): eight lanes have a unit each; neighbouring units of a page go as one copy.
template <int FMT, int D, bool QUAD>
__device__ __forceinline__ void rows_feed(const KvAttnArgs& a, uint8_t* smem, const RowBars& bar) {
    using C = RCfg<FMT, D, QUAD>;
    using U = typename C::U;
    const int lane = threadIdx.x & 31;
    const Plan plan = make_plan<kTokens, C::ROWS, C::EXTRA>(a, kMinRowTiles);
    if (lane == 0) reinterpret_cast<Split*>(a.partial)[blockIdx.x].parts = 0;
    int64_t at = plan.at, off = plan.off;
    const int64_t stop = min(at + plan.per, plan.work);
    int b = plan.b, qt = plan.qt;
    Seq s = plan.s;
    uint32_t tiles = 0;
#pragma unroll 1
    for (uint32_t nseg = 0;; ++nseg) {
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
            const TileSpan span = tile_span<kTokens, C::ROWS>(a, s.kv, s.qn, qt);
            t0 = span.first, n = span.count;
            const int64_t each = n + C::EXTRA;  // of a head
            if (off >= each * a.kv_heads) {
                off -= each * a.kv_heads;
                ++qt;
                continue;
            }
            head = div_small(off, each, place);
            share = min(each - place, stop - at);
            from = max(static_cast<int>(place) - C::EXTRA, 0);
            count = max(static_cast<int>(place + share) - C::EXTRA, 0) - from;
            if (count > 0) break;
            at += share;  // nothing but tiles that are only counted
            off += share;
        }
        if (!wait_warp(&bar.seg_empty[buf], (nseg >> 1 & 1u) ^ 1u, a.status, 0x51)) return;
        if (count == 0) {
            if (lane == 0) {
                note->count = -1;
                mbar_arrive(&bar.seg_full[buf]);
            }
            return;
        }
        const int row0 = qt * C::ROWS, rows = min(C::ROWS, s.qn * a.group - row0);
        int seen0, seen1, all0, all1;
        row_span(a, s, row0, seen0, all1);
        row_span(a, s, row0 + rows - 1, all0, seen1);
        if (lane == 0) {
            note->count = count;
            note->base = tiles;
            note->pos0 = (t0 + from) * kTokens;
            note->seen0 = seen0, note->seen1 = seen1, note->all0 = all0, note->all1 = all1;
            note->q0 = s.q0, note->row0 = row0, note->rows = rows, note->head = head;
            note->kv = s.kv, note->qn = s.qn;
            note->begins = from == 0;
            note->whole = from == 0 && count == n;
            int64_t rest;
            note->parts = from == 0 ? div_small(at - place + C::EXTRA + n - 1, plan.per, rest) - static_cast<int>(blockIdx.x) + 1 : 0;
            mbar_arrive(&bar.seg_full[buf]);
        }
        const int first_unit = (t0 + from) * C::UNITS;
        // In front of and behind the tokens that some row sees, pages may not exist (a window's may have been given away)
        const int units_from = seen0 >> 4, units_end = min((seen1 + 15) >> 4, first_unit + count * C::UNITS);
        auto source_of = [&](int i) -> int64_t {  // of the lane's unit of tile i; not loaded: -1, and -2 where the page is none of the cache's
            const int unit = first_unit + i * C::UNITS + lane;
            if (lane >= C::UNITS || unit < units_from || unit >= units_end) return -1;
            const int at_page = a.page_units == 1 ? unit : static_cast<int>(__umulhi(unit, a.page_magic));
            const int pg = a.table[static_cast<int64_t>(b) * a.table_stride + at_page];
            if (pg < 0 || pg >= a.num_pages) {
                kv_status(a.status, kStatusKvPage);
                return -2;
            }
            return (static_cast<int64_t>(pg) * a.kv_heads + head) * a.page_bytes +
                   static_cast<int64_t>(unit - at_page * a.page_units) * U::BYTES;
        };
        // a later segment's rows of Q, on their way while the last one is worked on
        for (int r = lane; nseg > 0 && r < rows; r += 32) {
            const int j = (row0 + r) / a.group;
            const __nv_bfloat16* src = a.q + static_cast<int64_t>(s.q0 + j) * a.q_token_stride +
                                  static_cast<int64_t>(head * a.group + row0 + r - j * a.group) * a.q_head_stride;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
            if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64));
        }
        __syncwarp();
        int64_t next = source_of(0);
#pragma unroll 1
        for (int i = 0; i < count; ++i, ++tiles) {
            const int64_t src = next;
            next = source_of(i + 1);
            const uint32_t slot = tiles % C::STAGES;
            if (!wait_warp(&bar.raw_empty[slot], (tiles / C::STAGES & 1u) ^ 1u, a.status, 0x52)) return;
            const uint32_t valid = __ballot_sync(0xffffffffu, src >= 0), skip = __ballot_sync(0xffffffffu, src == -2);
            const int64_t before = __shfl_up_sync(0xffffffffu, src, 1);
            const bool cont = lane > 0 && src >= 0 && before >= 0 && src == before + U::BYTES;
            const uint32_t conts = __ballot_sync(0xffffffffu, cont);
            if (lane == 0) {
                reinterpret_cast<uint32_t*>(smem + C::OFF_SKIP)[tiles & 7] = skip;  // (in front of the arrival)
                mbar_arrive_expect_tx(&bar.raw_full[slot], __popc(valid) * U::BYTES);
            }
            __syncwarp();
            if (src >= 0 && !cont) {
                const int run = __ffs(~(conts >> (lane + 1)));  // this unit and those that follow it without a gap
                bulk_load(smem + C::OFF_RAW + slot * C::RAW + lane * U::BYTES, a.cache + src, run * U::BYTES, &bar.raw_full[slot]);
            }
            __syncwarp();
        }
        at += share;
        off += share;
    }
}

// Issues the products (whole warp, one lane elected).
template <int FMT, int D, bool QUAD>
__device__ __forceinline__ void rows_mma(const KvAttnArgs& a, uint8_t* smem, const RowBars& bar, uint32_t tmem) {
    using C = RCfg<FMT, D, QUAD>;
    // kind::f16 with f16 (formats 0) or bf16 operands (formats 1), fp32 accumulator
    constexpr uint32_t KIND = (1u << 4) | (FMT == MXQ_MXFP4 ? 1u << 7 | 1u << 10 : 0u);
    constexpr uint32_t IDESC_S = KIND | ((kTokens >> 3) << 17) | ((128u >> 4) << 24);
    constexpr uint32_t IDESC_O = KIND | ((static_cast<uint32_t>(D) >> 3) << 17) | ((128u >> 4) << 24);
    const uint32_t q = smem_u32(smem + C::OFF_Q);
    auto product = [&](uint32_t t, bool first) -> bool {  // O += P V of tile t
        if (!wait_warp(&bar.vf[t & 1], t >> 1 & 1u, a.status, 0x53)) return false;
        if (!wait_warp(&bar.pf[t & 1], t >> 1 & 1u, a.status, 0x54)) return false;
        tc_fence_after();
        if (elect_one()) {
            const uint32_t v = smem_u32(smem + C::OFF_V + (t & 1) * C::V16);
#pragma unroll
            for (int j = 0; j < kTokens / 16; ++j) {
                const uint64_t vd = smem_desc(v + (j >> 2) * (D * 128) + (j & 3) * 32, 16, 1024, kLayoutSwizzle128B);
                const uint32_t o = tmem + C::O_COL + (t & 1) * D;
                const uint32_t p = tmem + C::S_COL + (t & 1) * 128 + (FMT == MXQ_MXFP4 ? (j >> 1) * 32 + (j & 1) * 8 : j * 8);
                mma_bf16_ts(o, p, vd, IDESC_O, first && j == 0 ? 0u : 1u);
                if constexpr (FMT == MXQ_MXFP4) mma_bf16_ts(o, p + 16, vd, IDESC_O, 1u);  // P's lower bits
            }
            tc_commit(&bar.od[t & 1]);
        }
        __syncwarp();
        return true;
    };
    uint32_t t = 0;
#pragma unroll 1
    for (uint32_t nseg = 0;; ++nseg) {
        const uint32_t buf = nseg & 1u;
        if (!wait_warp(&bar.seg_full[buf], nseg >> 1 & 1u, a.status, 0x55)) return;
        const int count = reinterpret_cast<const Segment*>(smem + C::OFF_SEG + buf * 64)->count;
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&bar.seg_empty[buf]);
        if (count < 0) return;
        if (!wait_warp(bar.qf, nseg & 1u, a.status, 0x56)) return;
#pragma unroll 1
        for (int i = 0; i <= count; ++i) {
            if (i < count) {
                if (!wait_warp(&bar.kf[t & 1], t >> 1 & 1u, a.status, 0x57)) return;
                // S takes the place of P of tile t - 2, whose product has to be done
                if (t >= 2 && !wait_warp(&bar.od[t & 1], (t - 2) >> 1 & 1u, a.status, 0x58)) return;
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t k = smem_u32(smem + C::OFF_K + (t & 1) * C::K16);
#pragma unroll
                    for (int j = 0; j < D / 16; ++j) {
                        const uint32_t at = (j >> 2) * (kTokens * 128) + (j & 3) * 32;
                        mma_bf16(tmem + C::S_COL + (t & 1) * 128, smem_desc(q + at, 16, 1024, kLayoutSwizzle128B),
                                 smem_desc(k + at, 16, 1024, kLayoutSwizzle128B), IDESC_S, j == 0 ? 0u : 1u);
                    }
                    tc_commit(&bar.sf[t & 1]);
                    mbar_arrive(&bar.sf[t & 1]);  // hands on what the feeding warp noted of the tile
                }
                __syncwarp();
            }
            // behind the scores of the next tile, so that its softmax need not wait for this product
            if (i > 0 && !product(t - 1, i <= 2)) return;
            if (i < count) ++t;
        }
    }
}

// MXFP4 scale codes of a token's key blocks, one a byte.
template <int D>
__device__ __forceinline__ uint32_t key_codes(uint32_t at) {
    if constexpr (D == 64) return ld_shared_u16(at);
    uint32_t x[1];
    lds<4>(at, x);
    return x[0];
}

// Keys of units u, u + 1: a lane has quarter q of token r: 32-bit words of 8 elements, 16 bytes each once
// decoded.  Eight neighbouring lanes have four tokens and two quarters, whose chunks meet different banks.
// `loaded` is called once the raw bytes are in registers; it waits for the operand's place.
template <int FMT, int D, bool QUAD, class Loaded>
__device__ __forceinline__ bool keys(uint32_t raw, uint32_t k16, int u, Loaded loaded) {
    using U = typename RCfg<FMT, D, QUAD>::U;
    const int lane = threadIdx.x & 31;
    const int r0 = (lane >> 3 & 1) * 4 + (lane >> 1 & 3), q = (lane >> 4) * 2 + (lane & 1);
    uint32_t sc[4], w[4][U::W / 4];  // loads first: a warp's own latency is what its tile takes
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t unit = raw + (u + i / 2) * U::BYTES;
        const int r = r0 + 8 * (i & 1);
        if constexpr (FMT == MXQ_NVFP4) {
            sc[i] = D == 128 ? ld_shared_u16(unit + U::OFF_KS + r * U::NB + 2 * q) : ld_shared_u8(unit + U::OFF_KS + r * U::NB + q);
        } else {
            sc[i] = key_codes<D>(unit + U::OFF_KS + r * U::NB);
        }
        lds<U::W>(unit + U::k_at(r, q, 0), w[i]);
    }
    if (!loaded()) return false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t row = u * 16 + 8 * i + r0;
        uint32_t f = 0;
        if constexpr (FMT == MXQ_NVFP4) f = e4m3x2_f16x2(sc[i]);
#pragma unroll
        for (int k = 0; k < U::W / 4; ++k) {
            uint32_t o[4], chunk;  // of the word's 8 elements; their place in the row
            if constexpr (FMT == MXQ_NVFP4) {
                const uint32_t f2 = k < 2 ? prmt(f, f, 0x1010u) : prmt(f, f, 0x3232u);
                chunk = q * (U::W / 4) + k;
                e2m1x8(w[i][k], o);
#pragma unroll
                for (int x = 0; x < 4; ++x) o[x] = hmul2(o[x], f2);
            } else {  // word k lies in block k
                const MxFactor<kKeyOffset> f2((sc[i] >> (8 * k) & 0xFFu) * 0x10001u);
                chunk = 4 * k + q;
                e2m1x8_tiny(w[i][k], o);
#pragma unroll
                for (int x = 0; x < 4; ++x) o[x] = f2.of(o[x]);
            }
            st_shared_v4(k16 + (chunk >> 3) * (kTokens * 128) + row * 128 + (((chunk & 7) ^ (r0 & 7)) << 4),
                         make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
    return true;
}

// Values of unit u, transposed: a lane has tokens 8 h + 2 t, + 1 and channels 16 j + 2 g, + 1.
template <int FMT, int D, bool QUAD, class Loaded>
__device__ __forceinline__ bool values(uint32_t raw, uint32_t v16, int u, bool edge, int pos0, int seen0, int seen1,
                                       const uint8_t* smem, uint32_t n, Loaded loaded) {
    using C = RCfg<FMT, D, QUAD>;
    using U = typename C::U;
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const uint32_t unit = raw + u * U::BYTES;
    // channel 16 j + 2 g has swizzle row 2 g, the next one 2 g + 1, whatever j is
    const uint32_t to = v16 + (u >> 2) * (D * 128) + 2 * g * 128 + 4 * t;
    constexpr int PB = 2 * U::NB;
    uint32_t sb[2][PB / 4], w[2][U::W / 4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        lds<PB>(unit + U::OFF_VS + (t + 4 * h) * PB, sb[h]);
        lds<U::W>(unit + U::OFF_V + h * (4 * D) + lane * U::W, w[h]);
    }
    if (!loaded()) return false;
    if (edge) {
        // tokens that no row sees: 0, whatever the bytes are; a NaN of E4M3 (the quantizer writes none): the largest
        // number, as 0 times it has to be 0 for the rows that do not see the token (E8M0's stands for 2^128 here)
        const uint32_t skip = skipped<C>(smem, n);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t live = skip >> u & 1u ? 0u : pair_mask(pos0 + 16 * u + 8 * h + 2 * t, seen0, seen1);
#pragma unroll
            for (int i = 0; i < PB / 4; ++i) {
                sb[h][i] &= live;
                if constexpr (FMT == MXQ_NVFP4) sb[h][i] = __vminu4(sb[h][i] & 0x7F7F7F7Fu, 0x7E7E7E7Eu);
            }
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t chunk = (u & 3) * 2 + h;  // of 8 tokens in the block of 64
        // lanes with g >= 4 take the odd channel first: else rows 2 g and 2 (g + 4) would meet the same banks
        const uint32_t even = to + ((chunk ^ (2 * g & 7)) << 4), odd = to + 128 + ((chunk ^ ((2 * g + 1) & 7)) << 4);
        const uint32_t at0 = g < 4 ? even : odd, at1 = g < 4 ? odd : even;
        auto scaled = [&](uint32_t x, int j) {  // of the two tokens, channel 16 j + ...
            const int b = FMT == MXQ_NVFP4 ? j : j / 2;
            if constexpr (FMT == MXQ_NVFP4)
                return hmul2(x, e4m3x2_f16x2(b & 1 ? sb[h][b >> 1] >> 16 : sb[h][b >> 1] & 0xFFFFu));
            else
                return MxFactor<kValueOffset>(prmt(sb[h][b >> 1], 0u, b & 1 ? 0x4342u : 0x4140u)).of(x);
        };
#pragma unroll
        for (int wd = 0; wd < D / 64; ++wd) {
            const uint32_t x = w[h][wd], y = w[h][D / 64 + wd];
            const uint32_t lo = (x & 0x0F0F0F0Fu) | (y << 4 & 0xF0F0F0F0u), hi = (x >> 4 & 0x0F0F0F0Fu) | (y & 0xF0F0F0F0u);
            uint32_t v0[4], v1[4];
            if constexpr (FMT == MXQ_NVFP4) {
                e2m1x8(g < 4 ? lo : hi, v0);
                e2m1x8(g < 4 ? hi : lo, v1);
            } else {
                e2m1x8_tiny(g < 4 ? lo : hi, v0);
                e2m1x8_tiny(g < 4 ? hi : lo, v1);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = 4 * wd + k;
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at0 + j * 2048), "r"(scaled(v0[k], j)) : "memory");
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at1 + j * 2048), "r"(scaled(v1[k], j)) : "memory");
            }
        }
    }
    return true;
}

template <int FMT>
__device__ __forceinline__ float score_scale(const KvAttnArgs& a) {
    float s = a.scale * 1.4426950408889634f;
    if constexpr (FMT == MXQ_NVFP4)
        s *= *a.g_k;
    else
        s *= static_cast<float>(1 << kKeyOffset);
    return s;
}

// Q rows of a segment, times a power of two (largest element in [2^7, 2^8)).  Of eight warps each takes every
// eighth row, all its lanes one row at a time; QUAD: the row stands in all four groups of lanes.
template <int FMT, int D, bool QUAD>
__device__ __forceinline__ void queries(const KvAttnArgs& a, const Segment& note, uint8_t* smem, float* qs, float qscale, int warp) {
    using C = RCfg<FMT, D, QUAD>;
    const int lane = threadIdx.x & 31;
    constexpr int WARPS = 8, PER = C::ROWS / WARPS, E = D / 32;  // rows of a warp, elements of a lane
    uint32_t x[PER < 8 ? PER : 8][E / 2];
#pragma unroll 1
    for (int k0 = 0; k0 < PER; k0 += 8) {
#pragma unroll
        for (int k = 0; k < 8 && k < PER; ++k) {
            const int rq = (k0 + k) * WARPS + warp, row = note.row0 + rq, j = row / a.group;
#pragma unroll
            for (int i = 0; i < E / 2; ++i) x[k][i] = 0;
            if (rq < note.rows) {
                const uint32_t* src = reinterpret_cast<const uint32_t*>(
                    a.q + static_cast<int64_t>(note.q0 + j) * a.q_token_stride +
                    static_cast<int64_t>(note.head * a.group + row - j * a.group) * a.q_head_stride + lane * E);
                if constexpr (E == 2) {
                    x[k][0] = *src;
                } else {
                    const uint2 y = *reinterpret_cast<const uint2*>(src);
                    x[k][0] = y.x, x[k][1] = y.y;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 8 && k < PER; ++k) {
            const int rq = (k0 + k) * WARPS + warp;
            uint32_t top = 0;  // bf16 magnitudes order like integers
#pragma unroll
            for (int i = 0; i < E / 2; ++i) top = __vmaxu2(top, x[k][i] & 0x7FFF7FFFu);
            const uint32_t ex = max(__reduce_max_sync(0xffffffffu, max(top & 0xFFFFu, top >> 16)) >> 7, 8u);
            const float mul = __uint_as_float((261u - ex) << 23);
            if (lane == 0) qs[rq] = qscale * __uint_as_float((ex - 7u) << 23);
            const int e = lane * E, c = e / 8;  // first element, its chunk of 8
#pragma unroll
            for (int copy = 0; copy < 128 / C::ROWS; ++copy) {
                const int tr = copy * C::ROWS + rq;
                uint32_t* dst = reinterpret_cast<uint32_t*>(smem + C::OFF_Q + (c >> 3) * (128 * 128) + tr * 128 +
                                                            (((c & 7) ^ (tr & 7)) << 4) + e % 8 * 2);
#pragma unroll
                for (int i = 0; i < E / 2; ++i)
                {
                    const float q0 = __uint_as_float(x[k][i] << 16) * mul, q1 = __uint_as_float(x[k][i] & 0xFFFF0000u) * mul;
                    // (bf16: exact, so its upper halves)
                    dst[i] = FMT == MXQ_MXFP4 ? prmt(__float_as_uint(q0), __float_as_uint(q1), 0x7632u) : cvt_f16x2(q0, q1);
                }
            }
        }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// Decodes tiles to 16-bit operands: warps 0-3 the keys of two units each, warps 4-11 the values of one.
template <int FMT, int D, bool QUAD>
__device__ __forceinline__ void rows_decode(const KvAttnArgs& a, uint8_t* smem, const RowBars& bar, int warp) {
    using C = RCfg<FMT, D, QUAD>;
    using U = typename C::U;
    const int lane = threadIdx.x & 31;
    const float qscale = QUAD ? 0.0f : score_scale<FMT>(a);
#pragma unroll 1
    for (uint32_t nseg = 0;; ++nseg) {
        const uint32_t buf = nseg & 1u;
        if (!wait_warp(&bar.seg_full[buf], nseg >> 1 & 1u, a.status, 0x59)) return;
        Segment note = *reinterpret_cast<const Segment*>(smem + C::OFF_SEG + buf * 64);
        const int count = note.count, seen0 = note.seen0, seen1 = note.seen1, all0 = note.all0, all1 = note.all1;
        const uint32_t base = note.base;
        int pos0 = note.pos0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.seg_empty[buf]);
        if (count < 0) return;
        // The value warps bring Q, beside the end of the segment before: its last scores are done when their
        // probabilities are written.  (In QUAD mode the softmax warps do, as their join lies where Q does.)
        if (!QUAD && warp >= kKeyWarps) {
            const uint32_t last = base - 1;
            if (nseg > 0 && !wait_warp(&bar.pf[last & 1], last >> 1 & 1u, a.status, 0x65)) return;
            queries<FMT, D, QUAD>(a, note, smem, reinterpret_cast<float*>(smem + C::OFF_QS) + buf * 128, qscale, warp - kKeyWarps);
            if (lane == 0) mbar_arrive(bar.qf);
        }
#pragma unroll 1
        for (int i = 0; i < count; ++i, pos0 += kTokens) {
            const uint32_t n = base + i, slot = n % C::STAGES;
            if (!wait_warp(&bar.raw_full[slot], n / C::STAGES & 1u, a.status, 0x5a)) return;
            const uint32_t raw = smem_u32(smem + C::OFF_RAW + slot * C::RAW);
            // the raw tile is given back as soon as it is in registers, then the operand's place waited for
            auto loaded = [&]() {
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.raw_empty[slot]);
                return warp < kKeyWarps ? wait_warp(&bar.sf[n & 1], (n >> 1 & 1u) ^ 1u, a.status, 0x5b)
                                        : wait_warp(&bar.od[n & 1], (n >> 1 & 1u) ^ 1u, a.status, 0x5c);
            };
            if (warp < kKeyWarps) {
                if (!keys<FMT, D, QUAD>(raw, smem_u32(smem + C::OFF_K + (n & 1) * C::K16), 2 * warp, loaded)) return;
            } else {
                if (!values<FMT, D, QUAD>(raw, smem_u32(smem + C::OFF_V + (n & 1) * C::V16), warp - kKeyWarps,
                                          skipped<C>(smem, n) != 0 || pos0 < all0 || pos0 + kTokens > all1, pos0, seen0, seen1, smem, n, loaded))
                    return;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(warp < kKeyWarps ? &bar.kf[n & 1] : &bar.vf[n & 1]);
        }
    }
}

// A value of O.
template <int FMT>
__device__ __forceinline__ float value(uint32_t x) {
    return FMT == MXQ_MXFP4 ? __uint_as_float(x) * static_cast<float>(1 << kValueOffset) : __uint_as_float(x);
}

// Softmax: a thread has one row (QUAD: one row and a quarter of each tile's tokens) in every second tile.
template <int FMT, int D, bool QUAD>
__device__ __forceinline__ void rows_softmax(const KvAttnArgs& a, uint8_t* smem, const RowBars& bar, uint32_t tmem) {
    using C = RCfg<FMT, D, QUAD>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = warp >> 2, quad = warp & 3;
    const int tl = quad * 32 + lane, r = QUAD ? lane : tl;          // TMEM lane, row
    const uint32_t lanes = tmem + (static_cast<uint32_t>(quad) << 21);  // the warp's 32 TMEM lanes
    constexpr int CHUNKS = QUAD ? 1 : 4;                                // of 32 tokens
    const int chunk0 = QUAD ? quad : 0;
    float* merge = reinterpret_cast<float*>(smem + C::OFF_Q);
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    float* partials = a.partial + gridDim.x * (sizeof(Split) / 4);
    const float gv = FMT == MXQ_NVFP4 ? *a.g_v : 1.0f;
    const float qscale = QUAD ? score_scale<FMT>(a) : 0.0f;
    uint32_t v[32];
#pragma unroll 1
    for (uint32_t nseg = 0;; ++nseg) {
        const uint32_t buf = nseg & 1u;
        bool dead = !wait_warp(&bar.seg_full[buf], nseg >> 1 & 1u, a.status, 0x5d);
        // one decision for all; also: the last segment's merge buffer, which Q overlies, has been read
        if (named_barrier_or(1, kSoftWarps * 32, dead)) return;
        const Segment note = *reinterpret_cast<const Segment*>(smem + C::OFF_SEG + buf * 64);
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.seg_empty[buf]);
        if (note.count < 0) return;
        float* qs = reinterpret_cast<float*>(smem + C::OFF_QS) + buf * 128;
        if constexpr (QUAD) {
            queries<FMT, D, QUAD>(a, note, smem, qs, qscale, warp);
            if (lane == 0) mbar_arrive(bar.qf);
        } else {
            dead = !wait_warp(bar.qf, nseg & 1u, a.status, 0x64);
        }
        // this thread's row
        int first = 0, end = 0;
        const bool real = r < note.rows;
        const int row = note.row0 + (real ? r : 0), jq = row / a.group;
        const int64_t orow = static_cast<int64_t>(note.q0 + jq) * a.heads + note.head * a.group + row - jq * a.group;
        {
            Seq s;
            s.kv = note.kv, s.q0 = note.q0, s.qn = note.qn;
            if (real) row_span(a, s, row, first, end);
        }
        if (named_barrier_or(1, kSoftWarps * 32, dead)) return;
        const float cs = qs[r];

        float base = kNegMax, l = 0.0f;
        const uint32_t o_at = lanes + C::O_COL + group * D;
        bool begun = false;  // O holds something
        // tiles n with n & 1 = group
#pragma unroll 1
        for (uint32_t n = note.base + ((note.base ^ group) & 1u); n < note.base + note.count; n += 2) {
            if (!wait_warp(&bar.sf[group], n >> 1 & 1u, a.status, 0x5e)) {
                dead = true;
                break;
            }
            tc_fence_after();
            const uint32_t s_at = lanes + C::S_COL + group * 128;
            const int pos0 = note.pos0 + static_cast<int>(n - note.base) * kTokens;
            const bool edge = skipped<C>(smem, n) != 0 || pos0 < note.all0 || pos0 + kTokens > note.all1;
#pragma unroll 1
            for (int c = chunk0; c < chunk0 + CHUNKS; ++c) {
                auto exponents = [&](float from) {  // of the chunk, relative to `from`; the largest
                    tmem_ld_32x32b_x32(s_at + 32 * c, v);
                    tmem_ld_wait();
                    float m0 = kNegMax, m1 = kNegMax;
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(fmaf(__uint_as_float(v[k]), cs, -from));
                    if (edge) {
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const int pos = pos0 + 32 * c + k;
                            if (pos < first || pos >= end) v[k] = 0xff800000u;
                        }
                        const uint32_t skip = skipped<C>(smem, n) >> (2 * c);
                        if (skip & 3u) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (skip >> (k / 16) & 1u) v[k] = 0xff800000u;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 32; k += 2) {
                        m0 = fmaxf(m0, __uint_as_float(v[k]));
                        m1 = fmaxf(m1, __uint_as_float(v[k + 1]));
                    }
                    return fmaxf(m0, m1);
                };
                const float m = exponents(base);
                if (__any_sync(0xffffffffu, m > kLimit || far_base(base))) {
                    // the product before the last of this group's tiles is done (its S was issued behind it); the tile's
                    // earlier P, which is read back below, is on its way: stores and loads of TMEM are not ordered
                    tmem_st_wait();
                    const float raw = exponents(0.0f);
                    // Bases are whole numbers, so that what is written already changes by a power of two, exactly, in
                    // l, O and P alike.  (A base at its start is far below; one that is no number makes the row none.)
                    const float to = raw - base > kLimit ? fmaxf(base, ceilf(raw - kStart)) : base, by = to - base;
                    const float al = by < 126.0f ? __uint_as_float(static_cast<uint32_t>(127 - static_cast<int>(by)) << 23) : 0.0f;
                    base = to;
                    l *= al;
                    if (begun) {
#pragma unroll 1
                        for (int k0 = 0; k0 < D; k0 += 32) {
                            tmem_ld_32x32b_x32(o_at + k0, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * al);
                            tmem_st_x16(o_at + k0, v);
                            tmem_st_x16(o_at + k0 + 16, v + 16);
                        }
                    }
                    if constexpr (FMT == MXQ_MXFP4) {
                        const uint32_t a2 = prmt(__float_as_uint(al), 0u, 0x3232u);
#pragma unroll 1
                        for (int c2 = 0; c2 < c; ++c2) {  // what the tile's P holds already
                            tmem_ld_32x32b_x32(s_at + 32 * c2, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[k] = bmul2(v[k], a2);
                            tmem_st_x16(s_at + 32 * c2, v);
                            tmem_st_x16(s_at + 32 * c2 + 16, v + 16);
                        }
                    } else {
                        // in two steps, as f16 has no factor below 2^-24
                        const float al_a = fmaxf(al, 0x1p-14f), al_b = fminf(al * 0x1p14f, 1.0f);
                        const uint32_t a2 = cvt_f16x2(al_a, al_a), b2 = cvt_f16x2(al_b, al_b);
#pragma unroll 1
                        for (int c2 = chunk0; c2 < c; ++c2) {
                            uint32_t p[16];
                            tmem_ld_32x32b_x16(s_at + 16 * c2, p);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k) p[k] = hmul2(hmul2(p[k], a2), b2);
                            tmem_st_x16(s_at + 16 * c2, p);
                        }
                    }
                    tmem_st_wait();
                    const float off = far_base(base) ? base : 0.0f;
                    exponents(base - off);
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(at_most(__uint_as_float(v[k]) - off, kLimit));
                }
                uint32_t p[FMT == MXQ_MXFP4 ? 32 : 16];
                float l0 = 0.0f, l1 = 0.0f;
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float e0 = ex2(__uint_as_float(v[2 * k])), e1 = ex2(__uint_as_float(v[2 * k + 1]));
                    l0 += e0;
                    l1 += e1;
                    if constexpr (FMT == MXQ_MXFP4) {  // the upper 8 bits, cut off, and the next 8, rounded: 2^-16 of e at most is lost
                        p[k] = prmt(__float_as_uint(e0), __float_as_uint(e1), 0x7632u);
                        const __nv_bfloat162 rest = __floats2bfloat162_rn(e0 - __uint_as_float(__float_as_uint(e0) & 0xFFFF0000u),
                                                                          e1 - __uint_as_float(__float_as_uint(e1) & 0xFFFF0000u));
                        p[16 + k] = *reinterpret_cast<const uint32_t*>(&rest);
                    } else {
                        p[k] = cvt_f16x2(e0, e1);
                    }
                }
                l += l0 + l1;
                if constexpr (FMT == MXQ_MXFP4) {
                    tmem_st_x16(s_at + 32 * c, p);
                    tmem_st_x16(s_at + 32 * c + 16, p + 16);
                } else {
                    tmem_st_x16(s_at + 16 * c, p);
                }
            }
            if constexpr (QUAD) {  // the other warps' tokens
                uint32_t z[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) z[k] = 0;
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (c != quad) tmem_st_x16(s_at + 16 * c, z);
            }
            begun = true;
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.pf[group]);
        }
        // the last products of both groups (each group has a tile, unless there is only one)
        const uint32_t last = note.base + note.count - 1;
        const bool both = note.count > 1;
        if (!dead) dead = !wait_warp(&bar.od[last & 1], last >> 1 & 1u, a.status, 0x60);
        if (!dead && both) dead = !wait_warp(&bar.od[(last - 1) & 1], (last - 1) >> 1 & 1u, a.status, 0x61);
        ml[group * 128 + tl] = make_float2(base, l);
        if (named_barrier_or(1, kSoftWarps * 32, dead)) return;
        tc_fence_after();
        float* part = partials + (static_cast<int64_t>(blockIdx.x) * 2 + (note.begins ? 1 : 0)) * (C::ROWS * (D + 2));
        if (note.begins && !note.whole && threadIdx.x == 0) {
            Split* split = reinterpret_cast<Split*>(a.partial) + blockIdx.x;
            split->parts = note.parts;
            split->q0 = note.q0;
            split->row0 = note.row0;
            split->rows = note.rows;
            split->head = note.head;
        }
        // this lane's O of both groups, weighted; a group without a tile has nothing (its columns are stale)
        const bool has0 = both || (last & 1) == 0, has1 = both || (last & 1) == 1;
        if constexpr (QUAD) {
            // Threads 8 jr .. 8 jr + 7 join row jr: of the eight results (two groups, four lanes), a slice of
            // the channels each; group 0 reads even slices from TMEM, group 1 odd ones, in turn.
            constexpr int SL = 32;  // channels of a slice
            const int jr = threadIdx.x >> 3, jc = (threadIdx.x & 7) * (SL / 8);
            const int jrow = note.row0 + (jr < note.rows ? jr : 0), jj = jrow / a.group;
            const int64_t o = static_cast<int64_t>(note.q0 + jj) * a.heads + note.head * a.group + jrow - jj * a.group;
            float most = kNegMax, sum = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) most = fmaxf(most, ml[k * 32 + jr].x);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum += ml[k * 32 + jr].y * ex2(ml[k * 32 + jr].x - most);
            float f[4];
#pragma unroll 1
            for (int pass = 0; pass < D / SL; ++pass) {
                float y[SL / 8];
#pragma unroll
                for (int k = 0; k < SL / 8; ++k) y[k] = 0.0f;
#pragma unroll 1
                for (int gg = 0; gg < 2; ++gg) {
                    if (gg == 0 ? !has0 : !has1) continue;
                    if (group == (pass & 1)) {
                        tmem_ld_32x32b_x32(lanes + C::O_COL + gg * D + pass * SL, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < SL; ++k) merge[tl * C::MERGE + k] = __uint_as_float(v[k]);
                    }
                    named_barrier_sync(1, kSoftWarps * 32);
#pragma unroll
                    for (int w = 0; w < 4; ++w) f[w] = ex2(ml[gg * 128 + w * 32 + jr].x - most);
#pragma unroll
                    for (int k = 0; k < SL / 8; ++k)
#pragma unroll
                        for (int w = 0; w < 4; ++w) y[k] = fmaf(merge[(w * 32 + jr) * C::MERGE + jc + k], f[w], y[k]);
                    named_barrier_sync(1, kSoftWarps * 32);
                }
                const int d = SL * pass + jc;
                const float inv = gv * (sum > 0.0f ? 1.0f / sum : sum);
                if (note.whole) {
                    if (jr < note.rows) {
                        put4(a, o * D + d, y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv);
                        if (a.lse && d == 0)
                            a.lse[o] = sum == 0.0f ? __int_as_float(0xff800000) : (most + log2f(sum)) * 0.6931471805599453f;
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < SL / 8; ++k) part[jr * D + d + k] = y[k];
                    if (d == 0) *reinterpret_cast<float2*>(part + C::ROWS * D + 2 * jr) = make_float2(most, sum);
                }
            }
        } else {
            // each group takes half of the channels
            const float2 z0 = ml[tl], z1 = ml[128 + tl];
            const float most = fmaxf(z0.x, z1.x), f0 = has0 ? ex2(z0.x - most) : 0.0f, f1 = has1 ? ex2(z1.x - most) : 0.0f;
            const float sum = z0.y * f0 + z1.y * f1;
            const float inv = note.whole ? gv * (sum > 0.0f ? 1.0f / sum : sum) : 1.0f;
#pragma unroll 1
            for (int d = group * (D / 2); d < (group + 1) * (D / 2); d += 16) {
                float y[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) y[k] = 0.0f;
                uint32_t x[16];
                if (has0) {
                    tmem_ld_32x32b_x16(lanes + C::O_COL + d, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) y[k] = value<FMT>(x[k]) * f0;
                }
                if (has1) {
                    tmem_ld_32x32b_x16(lanes + C::O_COL + D + d, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k) y[k] = fmaf(value<FMT>(x[k]), f1, y[k]);
                }
                if (note.whole) {
                    if (real) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) y[k] *= inv;
                        put8(a, orow * D + d, y);
                        put8(a, orow * D + d + 8, y + 8);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) part[(d + k) * C::ROWS + r] = y[k];  // channel by channel: whole sectors
                }
            }
            if (group == 0) {
                if (!note.whole)
                    *reinterpret_cast<float2*>(part + C::ROWS * D + 2 * r) = make_float2(most, sum);
                else if (a.lse && real)
                    a.lse[orow] = sum == 0.0f ? __int_as_float(0xff800000) : (most + log2f(sum)) * 0.6931471805599453f;
            }
        }
        tc_fence_before();
    }
}

template <int FMT, int D, bool QUAD>
__global__ void __launch_bounds__(kRowThreads, 1) kv_attention_rows_kernel(const __grid_constant__ KvAttnArgs a) {
    using C = RCfg<FMT, D, QUAD>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const RowBars bar(smem + C::OFF_BAR, C::STAGES);
    uint32_t* slot = reinterpret_cast<uint32_t*>(smem + C::OFF_TMEM);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::STAGES; ++i) {
            mbar_init(&bar.raw_full[i], 1);
            mbar_init(&bar.raw_empty[i], kDecWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.kf[i], kKeyWarps);
            mbar_init(&bar.vf[i], kValueWarps);
            mbar_init(&bar.sf[i], 2);  // the products' end, and the issuing lane
            mbar_init(&bar.pf[i], kSoftWarps / 2);
            mbar_init(&bar.od[i], 1);
            mbar_init(&bar.seg_full[i], 1);
            mbar_init(&bar.seg_empty[i], kSoftWarps + kDecWarps + 1);
        }
        mbar_init(bar.qf, 8);  // softmax warps or value warps
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *slot;
    pdl_launch_dependents();
    pdl_wait();
    if (warp < kSoftWarps) {
        rows_softmax<FMT, D, QUAD>(a, smem, bar, tmem);
    } else if (warp < kFeedWarp) {
        rows_decode<FMT, D, QUAD>(a, smem, bar, warp - kSoftWarps);
    } else if (warp == kFeedWarp) {
        rows_feed<FMT, D, QUAD>(a, smem, bar);
    } else {
        rows_mma<FMT, D, QUAD>(a, smem, bar, tmem);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int FMT, int D, bool QUAD>
int run_rows(KvAttnArgs& a, cudaStream_t st) {
    using C = RCfg<FMT, D, QUAD>;
    static_assert(C::BYTES <= 227 * 1024, "shared memory");
    auto kernel = kv_attention_rows_kernel<FMT, D, QUAD>;
    auto join = kv_attention_join_kernel<FMT, D, C::ROWS>;
    static std::atomic<int> known[64];
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MXQ_ERR_CUDA;
    if (known[dev].load() == 0) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::BYTES) != cudaSuccess) return MXQ_ERR_CUDA;
        known[dev].store(1);
    }
    const int grid = std::min(sm_count(), kMaxGrid);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kRowThreads);
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

}  // namespace

int kv_rows_tile(int64_t rows) { return rows <= 32 ? 32 : 128; }

int launch_kv_attention_rows(int fmt, int D, KvAttnArgs& a, cudaStream_t st) {
    const bool quad = kv_rows_tile(static_cast<int64_t>(a.max_q) * a.group) == 32;
    if (fmt == MXQ_MXFP4) return D == 64 ? run_rows<MXQ_MXFP4, 64, false>(a, st) : run_rows<MXQ_MXFP4, 128, false>(a, st);
    if (D == 64) return run_rows<MXQ_NVFP4, 64, false>(a, st);
    return quad ? run_rows<MXQ_NVFP4, 128, true>(a, st) : run_rows<MXQ_NVFP4, 128, false>(a, st);
}

}  // namespace mxq
