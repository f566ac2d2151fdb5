// kv_cache.cu -- writing tokens into the 4-bit key/value cache (append) and reading them back.
#include "kv.cuh"
#include "kv_internal.h"
#include "mxq_internal.h"
#include "quant_block.cuh"

namespace mxq {
namespace {

constexpr int kThreads = 256;

// A warp takes 32 / (D / 32) consecutive tokens of one head and side, a lane 32 elements (chunk c) of one
// of them.  Consecutive tokens mostly have consecutive slots: then the warp's stores cover whole sectors of
// the unit (a warp over the heads of one token wrote 2-byte pieces of eight units: append and read of 8192
// tokens of 8 x 128 in MXFP4 took 31.0 us, this way round 26.2 us).
struct Place {
    uint32_t token, side, head, c;
    bool any;  // the token exists
};

template <int D>
__device__ __forceinline__ Place place_of(uint32_t tokens, uint32_t heads) {
    constexpr uint32_t CH = D / 32, PER = 32 / CH;
    const uint32_t w = (blockIdx.x * kThreads + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    const uint32_t hs = w % (2 * heads);
    Place p;
    p.token = w / (2 * heads) * PER + lane / CH;
    p.side = hs / heads;
    p.head = hs - p.side * heads;
    p.c = lane % CH;
    p.any = p.token < tokens;
    return p;
}

// V bytes change hands through shared memory: lane c of a row has byte g of the 16-element pieces 2c and
// 2c + 1 for all g; the cache wants, for each g, the bytes of all pieces together (D / 16 of them).
template <int D>
struct Exchange {
    static constexpr int ROW = D / 2 + 8;  // bytes; the skew keeps the rows' 2-byte accesses in different banks
    static constexpr int PIECE = D / 16;   // bytes of one g
    uint8_t at[kThreads / 32][32 / (D / 32)][ROW];
};

// bf16 values change hands through shared memory too: memory is read and written 16 bytes a lane, side by
// side, while a lane works on 64 contiguous ones (loading those itself, it touched every 32-byte sector
// twice: 26.2 us for append and read of 8192 tokens, 25.4 us so).  The warp's 2 KB are 128 pieces of 16 bytes, lane l's own
// being 4 l .. 4 l + 3; piece p lies at p ^ (p / 8 & 3), so that neither way meets a bank twice.
struct Pieces {
    uint4 at[kThreads / 32][128];
};
__device__ __forceinline__ int piece_at(int p) { return p ^ (p >> 3 & 3); }

// Appending: quantize with the arithmetic of the streaming quantizer and store codes and scales at the
// token's place in its unit.  Bound: HBM (2 D values read in bf16, written in 4 bits, per token and head).
template <int FMT, int RULE, int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a) {
    using U = KvUnit<FMT, D>;
    __shared__ float tabs[FMT == MXQ_NVFP4 ? 4 : 1][128];
    __shared__ __align__(8) Exchange<D> ex;
    __shared__ Pieces pieces;
    pdl_launch_dependents();
    pdl_wait();
    const Place p = place_of<D>(a.tokens, a.heads);
    const uint32_t c = p.c, side = p.side, lane = threadIdx.x & 31;
    int slot = p.any ? a.slots[p.token] : -1;
    {
        constexpr int ROW = D / 8;  // pieces of a token
        uint4* mine = pieces.at[threadIdx.x >> 5];
        const uint32_t token0 = p.token - lane / (D / 32);
        const __nv_bfloat16* src = (side ? a.v : a.k) + static_cast<int64_t>(p.head) * a.head_stride[side];
        uint4 x[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t i = q * 32 + lane, token = token0 + i / ROW;
            x[q] = make_uint4(0, 0, 0, 0);
            if (token < a.tokens)
                x[q] = __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(token) * a.token_stride[side]) + i % ROW);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) mine[piece_at(q * 32 + lane)] = x[q];
    }
    float g[2] = {1.0f, 1.0f};
    if constexpr (FMT == MXQ_NVFP4) {
        g[0] = *a.g_k;
        g[1] = *a.g_v;
        nvfp4_tables(g[0], tabs[0], tabs[1]);
        nvfp4_tables(g[1], tabs[2], tabs[3]);
        __syncthreads();
    }
    if (slot >= a.num_slots) {
        kv_status(a.status, kStatusKvSlot);
        slot = -1;
    }
    __syncwarp();
    uint32_t w[16], codes[4] = {0, 0, 0, 0}, seen = 0, sf = 0;
    if (slot >= 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 x = pieces.at[threadIdx.x >> 5][piece_at(4 * lane + q)];
            w[4 * q] = x.x;
            w[4 * q + 1] = x.y;
            w[4 * q + 2] = x.z;
            w[4 * q + 3] = x.w;
        }
        sf = quantize32<FMT, RULE, false>(w, g[side], tabs[FMT == MXQ_NVFP4 ? 2 * side : 0],
                                          tabs[FMT == MXQ_NVFP4 ? 2 * side + 1 : 0], codes, seen);
    }
    const uint32_t page = static_cast<uint32_t>(slot) / a.page_size, off = static_cast<uint32_t>(slot) % a.page_size;
    uint8_t* unit = a.cache + (static_cast<int64_t>(page) * a.heads + p.head) * a.page_bytes +
                    static_cast<int64_t>(off >> 4) * U::BYTES;
    const int r = off & 15;
    if (side == 0) {  // the same for the whole warp
        if (slot < 0) return;
        if constexpr (FMT == MXQ_NVFP4) {
            // row bytes [16 c, 16 c + 16): quarter and place inside follow from the quarter's D / 8 bytes
            const int t = static_cast<int>(c) * 16 / (D / 8), inside = static_cast<int>(c) * 16 % (D / 8);
            *reinterpret_cast<uint4*>(unit + U::k_at(r, t, inside)) = make_uint4(codes[0], codes[1], codes[2], codes[3]);
            *reinterpret_cast<uint16_t*>(unit + U::ks_at(r, 2 * c)) = static_cast<uint16_t>(sf);
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) *reinterpret_cast<uint32_t*>(unit + U::k_at(r, t, 4 * c)) = codes[t];
            unit[U::ks_at(r, c)] = static_cast<uint8_t>(sf);
        }
        return;
    }
    using X = Exchange<D>;
    uint8_t* row = ex.at[threadIdx.x >> 5][(threadIdx.x & 31) / (D / 32)];
#pragma unroll
    for (int q = 0; q < 2; ++q) {  // g = 4 q .. 4 q + 3: bytes (2c, g) and (2c + 1, g) side by side
        const uint32_t lo = prmt(codes[q], codes[2 + q], 0x5140u), hi = prmt(codes[q], codes[2 + q], 0x7362u);
        *reinterpret_cast<uint16_t*>(row + (4 * q) * X::PIECE + 2 * c) = static_cast<uint16_t>(lo);
        *reinterpret_cast<uint16_t*>(row + (4 * q + 1) * X::PIECE + 2 * c) = static_cast<uint16_t>(lo >> 16);
        *reinterpret_cast<uint16_t*>(row + (4 * q + 2) * X::PIECE + 2 * c) = static_cast<uint16_t>(hi);
        *reinterpret_cast<uint16_t*>(row + (4 * q + 3) * X::PIECE + 2 * c) = static_cast<uint16_t>(hi >> 16);
    }
    __syncwarp();
    if (slot < 0) return;
    const uint2 y0 = *reinterpret_cast<const uint2*>(row + 16 * c), y1 = *reinterpret_cast<const uint2*>(row + 16 * c + 8);
    if constexpr (D == 64) {
        *reinterpret_cast<uint32_t*>(unit + U::v_at(r, 4 * c, 0)) = y0.x;
        *reinterpret_cast<uint32_t*>(unit + U::v_at(r, 4 * c + 1, 0)) = y0.y;
        *reinterpret_cast<uint32_t*>(unit + U::v_at(r, 4 * c + 2, 0)) = y1.x;
        *reinterpret_cast<uint32_t*>(unit + U::v_at(r, 4 * c + 3, 0)) = y1.y;
    } else if constexpr (D == 128) {
        *reinterpret_cast<uint2*>(unit + U::v_at(r, 2 * c, 0)) = y0;
        *reinterpret_cast<uint2*>(unit + U::v_at(r, 2 * c + 1, 0)) = y1;
    } else {
        *reinterpret_cast<uint4*>(unit + U::v_at(r, c, 0)) = make_uint4(y0.x, y0.y, y1.x, y1.y);
    }
    if constexpr (FMT == MXQ_NVFP4) {
        unit[U::vs_at(r, 2 * c)] = static_cast<uint8_t>(sf);
        unit[U::vs_at(r, 2 * c + 1)] = static_cast<uint8_t>(sf >> 8);
    } else {
        unit[U::vs_at(r, c)] = static_cast<uint8_t>(sf);
    }
}

// Reading back, the same way round: elements times scale as fake quantization rounds them (MX exact, NVFP4
// fl32(elem * fl32(dec(s) * g)), then bf16).  A negative slot gives zeros.
template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadArgs a) {
    using U = KvUnit<FMT, D>;
    using X = Exchange<D>;
    __shared__ __align__(8) X ex;
    __shared__ Pieces pieces;
    pdl_launch_dependents();
    pdl_wait();
    const Place p = place_of<D>(a.tokens, a.heads);
    const uint32_t c = p.c, side = p.side;
    int slot = p.any ? a.slots[p.token] : -1;
    if (slot >= a.num_slots) {
        kv_status(a.status, kStatusKvSlot);
        slot = -1;
    }
    const uint32_t page = static_cast<uint32_t>(slot) / a.page_size, off = static_cast<uint32_t>(slot) % a.page_size;
    const uint8_t* unit = a.cache + (static_cast<int64_t>(page) * a.heads + p.head) * a.page_bytes +
                          static_cast<int64_t>(off >> 4) * U::BYTES;
    const int r = off & 15;
    uint32_t codes[4] = {0, 0, 0, 0};
    float d[2] = {0.0f, 0.0f};
    if (slot >= 0) {
        if constexpr (FMT == MXQ_NVFP4) {
            const float g = side ? *a.g_v : *a.g_k;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                d[b] = __fmul_rn(e4m3_decode_pos(unit[side ? U::vs_at(r, 2 * c + b) : U::ks_at(r, 2 * c + b)]), g);
        } else {
            d[0] = d[1] = pow2f(static_cast<int>(unit[side ? U::vs_at(r, c) : U::ks_at(r, c)]) - 127);
        }
    }
    if (side == 0) {
        if (slot >= 0) {
            if constexpr (FMT == MXQ_NVFP4) {
                const int t = static_cast<int>(c) * 16 / (D / 8), inside = static_cast<int>(c) * 16 % (D / 8);
                const uint4 x = *reinterpret_cast<const uint4*>(unit + U::k_at(r, t, inside));
                codes[0] = x.x, codes[1] = x.y, codes[2] = x.z, codes[3] = x.w;
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t) codes[t] = *reinterpret_cast<const uint32_t*>(unit + U::k_at(r, t, 4 * c));
            }
        }
    } else {
        uint8_t* row = ex.at[threadIdx.x >> 5][(threadIdx.x & 31) / (D / 32)];
        uint2 y0 = make_uint2(0, 0), y1 = make_uint2(0, 0);
        if (slot >= 0) {
            if constexpr (D == 64) {
                y0.x = *reinterpret_cast<const uint32_t*>(unit + U::v_at(r, 4 * c, 0));
                y0.y = *reinterpret_cast<const uint32_t*>(unit + U::v_at(r, 4 * c + 1, 0));
                y1.x = *reinterpret_cast<const uint32_t*>(unit + U::v_at(r, 4 * c + 2, 0));
                y1.y = *reinterpret_cast<const uint32_t*>(unit + U::v_at(r, 4 * c + 3, 0));
            } else if constexpr (D == 128) {
                y0 = *reinterpret_cast<const uint2*>(unit + U::v_at(r, 2 * c, 0));
                y1 = *reinterpret_cast<const uint2*>(unit + U::v_at(r, 2 * c + 1, 0));
            } else {
                const uint4 y = *reinterpret_cast<const uint4*>(unit + U::v_at(r, c, 0));
                y0 = make_uint2(y.x, y.y);
                y1 = make_uint2(y.z, y.w);
            }
        }
        *reinterpret_cast<uint2*>(row + 16 * c) = y0;
        *reinterpret_cast<uint2*>(row + 16 * c + 8) = y1;
        __syncwarp();
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = *reinterpret_cast<const uint16_t*>(row + (4 * q + k) * X::PIECE + 2 * c);
            const uint32_t lo = prmt(h[0], h[1], 0x5410u), hi = prmt(h[2], h[3], 0x5410u);  // halves (2c, 2c + 1) of g, g + 1
            codes[q] = prmt(lo, hi, 0x6420u);
            codes[2 + q] = prmt(lo, hi, 0x7531u);
        }
    }
    uint4* mine = pieces.at[threadIdx.x >> 5];
    const uint32_t lane = threadIdx.x & 31;
#pragma unroll
    for (int q = 0; q < 4; ++q) mine[piece_at(4 * lane + q)] = dequant8_cvt(codes[q], d[q >> 1]);
    __syncwarp();
    constexpr int ROW = D / 8;  // pieces of a token
    const uint32_t token0 = p.token - lane / (D / 32);
    __nv_bfloat16* dst = (side ? a.v_out : a.k_out) + static_cast<int64_t>(p.head) * D;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint32_t i = q * 32 + lane, token = token0 + i / ROW;
        if (token < a.tokens)
            reinterpret_cast<uint4*>(dst + static_cast<int64_t>(token) * a.heads * D)[i % ROW] = mine[piece_at(i)];
    }
}

template <typename K, typename A>
int launch(K kernel, uint32_t blocks, const A& a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? MXQ_OK : MXQ_ERR_CUDA;
}

uint32_t blocks_for(uint32_t tokens, uint32_t heads, int D) {
    const int64_t warps = ceil_div(tokens, 32 / (D / 32)) * 2 * heads;
    return static_cast<uint32_t>(ceil_div(warps * 32, kThreads));
}

template <int FMT, int RULE>
int append_dim(int D, const KvAppendArgs& a, cudaStream_t st) {
    const uint32_t n = blocks_for(a.tokens, a.heads, D);
    switch (D) {
        case 64: return launch(kv_append_kernel<FMT, RULE, 64>, n, a, st);
        case 128: return launch(kv_append_kernel<FMT, RULE, 128>, n, a, st);
        default: return launch(kv_append_kernel<FMT, RULE, 256>, n, a, st);
    }
}

template <int FMT>
int read_dim(int D, const KvReadArgs& a, cudaStream_t st) {
    const uint32_t n = blocks_for(a.tokens, a.heads, D);
    switch (D) {
        case 64: return launch(kv_read_kernel<FMT, 64>, n, a, st);
        case 128: return launch(kv_read_kernel<FMT, 128>, n, a, st);
        default: return launch(kv_read_kernel<FMT, 256>, n, a, st);
    }
}

}  // namespace

int launch_kv_append(int fmt, int rule, int D, const KvAppendArgs& a, cudaStream_t st) {
    if (fmt == MXQ_NVFP4) return append_dim<MXQ_NVFP4, MXQ_RULE_EVEN>(D, a, st);
    return rule == MXQ_RULE_CEIL ? append_dim<MXQ_MXFP4, MXQ_RULE_CEIL>(D, a, st)
                                 : append_dim<MXQ_MXFP4, MXQ_RULE_EVEN>(D, a, st);
}

int launch_kv_read(int fmt, int D, const KvReadArgs& a, cudaStream_t st) {
    return fmt == MXQ_NVFP4 ? read_dim<MXQ_NVFP4>(D, a, st) : read_dim<MXQ_MXFP4>(D, a, st);
}

}  // namespace mxq
