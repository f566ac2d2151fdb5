// kv_cache.cu -- writing tokens into the 4-bit key/value cache (append) and reading them back.
#include "kv.cuh"
#include "kv_internal.h"
#include "mxq_internal.h"
#include "quant_block.cuh"

namespace mxq {
namespace {

constexpr int kThreads = 256;

// Appending.  One thread quantizes 32 elements (one MX block or two NVFP4 blocks) of one token, head
// and side with the arithmetic of the streaming quantizer, and stores codes and scales at the token's
// place in its unit.  Bound: HBM (2 D values read in bf16, written in 4 bits, per token and head).
template <int FMT, int RULE, int D>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a) {
    using U = KvUnit<FMT, D>;
    __shared__ float tabs[FMT == MXQ_NVFP4 ? 4 : 1][128];
    pdl_launch_dependents();
    pdl_wait();
    float g[2] = {1.0f, 1.0f};
    if constexpr (FMT == MXQ_NVFP4) {
        g[0] = *a.g_k;
        g[1] = *a.g_v;
        nvfp4_tables(g[0], tabs[0], tabs[1]);
        nvfp4_tables(g[1], tabs[2], tabs[3]);
        __syncthreads();
    }
    constexpr uint32_t CH = D / 32;  // 32-element chunks of a row
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t c = i % CH, row = i / CH;  // row = (token * 2 + side) * heads + head
    const uint32_t head = row % a.heads, ts = row / a.heads;
    const uint32_t side = ts & 1u, token = ts >> 1;
    if (token >= a.tokens) return;
    const int slot = a.slots[token];
    if (slot < 0) return;
    if (slot >= a.num_slots) {
        kv_status(a.status, kStatusKvSlot);
        return;
    }
    const __nv_bfloat16* src = (side ? a.v : a.k) + static_cast<int64_t>(token) * a.token_stride[side] +
                               static_cast<int64_t>(head) * a.head_stride[side] + c * 32;
    uint32_t w[16];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(src) + q);
        w[4 * q] = x.x;
        w[4 * q + 1] = x.y;
        w[4 * q + 2] = x.z;
        w[4 * q + 3] = x.w;
    }
    uint32_t codes[4], seen = 0;
    const uint32_t sf =
        quantize32<FMT, RULE, false>(w, g[side], tabs[FMT == MXQ_NVFP4 ? 2 * side : 0],
                                     tabs[FMT == MXQ_NVFP4 ? 2 * side + 1 : 0], codes, seen);
    const uint32_t page = static_cast<uint32_t>(slot) / a.page_size, off = static_cast<uint32_t>(slot) % a.page_size;
    uint8_t* unit = a.cache + (static_cast<int64_t>(page) * a.heads + head) * a.page_bytes +
                    static_cast<int64_t>(off >> 4) * U::BYTES;
    const int r = off & 15;
    if (side == 0) {
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
    } else {
#pragma unroll
        for (int gg = 0; gg < 8; ++gg) {
            const uint32_t lo = codes[gg >> 2] >> (8 * (gg & 3)) & 0xFFu;        // j = 2 c
            const uint32_t hi = codes[2 + (gg >> 2)] >> (8 * (gg & 3)) & 0xFFu;  // j = 2 c + 1
            *reinterpret_cast<uint16_t*>(unit + U::v_at(r, gg, 2 * c)) = static_cast<uint16_t>(lo | hi << 8);
        }
        if constexpr (FMT == MXQ_NVFP4) {
            unit[U::vs_at(r, 2 * c)] = static_cast<uint8_t>(sf);
            unit[U::vs_at(r, 2 * c + 1)] = static_cast<uint8_t>(sf >> 8);
        } else {
            unit[U::vs_at(r, c)] = static_cast<uint8_t>(sf);
        }
    }
}

// Reading back: the same division of work; elements times scale as fake quantization rounds them
// (MX exact, NVFP4 fl32(elem * fl32(dec(s) * g)), then bf16).  A negative slot gives zeros.
template <int FMT, int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvReadArgs a) {
    using U = KvUnit<FMT, D>;
    pdl_launch_dependents();
    pdl_wait();
    constexpr uint32_t CH = D / 32;
    const uint32_t i = blockIdx.x * kThreads + threadIdx.x;
    const uint32_t c = i % CH, row = i / CH;
    const uint32_t head = row % a.heads, ts = row / a.heads;
    const uint32_t side = ts & 1u, token = ts >> 1;
    if (token >= a.tokens) return;
    int slot = a.slots[token];
    if (slot >= a.num_slots) {
        kv_status(a.status, kStatusKvSlot);
        slot = -1;
    }
    uint4 o[4];
    if (slot < 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = make_uint4(0, 0, 0, 0);
    } else {
        const uint32_t page = static_cast<uint32_t>(slot) / a.page_size, off = static_cast<uint32_t>(slot) % a.page_size;
        const uint8_t* unit = a.cache + (static_cast<int64_t>(page) * a.heads + head) * a.page_bytes +
                              static_cast<int64_t>(off >> 4) * U::BYTES;
        const int r = off & 15;
        uint32_t codes[4];
        if (side == 0) {
            if constexpr (FMT == MXQ_NVFP4) {
                const int t = static_cast<int>(c) * 16 / (D / 8), inside = static_cast<int>(c) * 16 % (D / 8);
                const uint4 x = *reinterpret_cast<const uint4*>(unit + U::k_at(r, t, inside));
                codes[0] = x.x, codes[1] = x.y, codes[2] = x.z, codes[3] = x.w;
            } else {
#pragma unroll
                for (int t = 0; t < 4; ++t) codes[t] = *reinterpret_cast<const uint32_t*>(unit + U::k_at(r, t, 4 * c));
            }
        } else {
            codes[0] = codes[1] = codes[2] = codes[3] = 0;
#pragma unroll
            for (int gg = 0; gg < 8; ++gg) {
                const uint32_t x = *reinterpret_cast<const uint16_t*>(unit + U::v_at(r, gg, 2 * c));
                codes[gg >> 2] |= (x & 0xFFu) << (8 * (gg & 3));
                codes[2 + (gg >> 2)] |= (x >> 8) << (8 * (gg & 3));
            }
        }
        float d[2];
        if constexpr (FMT == MXQ_NVFP4) {
            const float g = side ? *a.g_v : *a.g_k;
#pragma unroll
            for (int b = 0; b < 2; ++b)
                d[b] = __fmul_rn(e4m3_decode_pos(unit[side ? U::vs_at(r, 2 * c + b) : U::ks_at(r, 2 * c + b)]), g);
        } else {
            d[0] = d[1] = pow2f(static_cast<int>(unit[side ? U::vs_at(r, c) : U::ks_at(r, c)]) - 127);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = dequant8_cvt(codes[q], d[q >> 1]);
    }
    uint4* dst = reinterpret_cast<uint4*>((side ? a.v_out : a.k_out) + (static_cast<int64_t>(token) * a.heads + head) * D + c * 32);
#pragma unroll
    for (int q = 0; q < 4; ++q) dst[q] = o[q];
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
    return static_cast<uint32_t>(ceil_div(static_cast<int64_t>(tokens) * 2 * heads * (D / 32), kThreads));
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
