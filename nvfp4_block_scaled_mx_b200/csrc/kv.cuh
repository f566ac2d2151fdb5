// kv.cuh -- the byte layout of the 4-bit key/value cache, shared by the kernels that write it (append),
// read it back and attend over it.
//
// A layer is [pages][kv_heads][page_size / 16][unit].  A unit holds 16 tokens of one head and is laid
// out so that the attention kernel's warps read matrix-instruction operands with full-width,
// conflict-free shared-memory loads and no shuffles:
//   K codes  8 D bytes.  Lane (g, t) = (lane / 4, lane % 4) owns quarter t (D / 8 bytes) of tokens g and
//            g + 8 -- a row of the m16n8k16 A operand with the k index dealt so that a lane's codes are
//            contiguous.  NVFP4: quarter t is the t-th contiguous piece, so that a lane needs one scale
//            per 8 bytes; MXFP4: the 32-bit words t, t + 4, ..., so that each word of a lane lies in
//            another 32-block and the block's scale can be applied to the accumulator.
//            Stored [piece][token][t], pieces of W = min(16, D / 8) bytes.
//   V codes  8 D bytes.  Lane (g, t) owns the tokens 2t, 2t + 1 of each group of eight and, of each 16
//            elements j, byte g (elements 16 j + 2 g, + 1): the A operand of O^T = V^T P^T.  A token's
//            D / 16 bytes follow the other's.  Stored [token / 8][piece][lane].
//   K scales [token][nb].    V scales [token / 2][nb][token % 2].
#pragma once

#include "dequant.cuh"
#include "mxq_device.cuh"

namespace mxq {

template <int FMT, int D>
struct KvUnit {
    static constexpr int BS = FMT == MXQ_NVFP4 ? 16 : 32;
    static constexpr int NB = D / BS;               // scale bytes of one token and side
    static constexpr int W = D / 8 < 16 ? D / 8 : 16;  // piece bytes
    static constexpr int PIECES = (D / 8) / W;
    static constexpr int OFF_V = 8 * D;
    static constexpr int OFF_KS = 16 * D;
    static constexpr int OFF_VS = 16 * D + 16 * NB;
    static constexpr int BYTES = 16 * D + 32 * NB;

    // byte `inside` (0 .. D/8 - 1) of quarter t of token r's K row
    static __host__ __device__ constexpr int k_at(int r, int t, int inside) {
        return (inside / W) * (64 * W) + (r * 4 + t) * W + inside % W;
    }
    // byte j of lane group g of token r's V row (elements 16 j + 2 g, 16 j + 2 g + 1)
    static __host__ __device__ constexpr int v_at(int r, int g, int j) {
        const int inside = (r & 1) * (D / 16) + j;
        return OFF_V + (r >> 3) * (4 * D) + (inside / W) * (32 * W) + (4 * g + ((r & 7) >> 1)) * W + inside % W;
    }
    static __host__ __device__ constexpr int ks_at(int r, int b) { return OFF_KS + r * NB + b; }
    static __host__ __device__ constexpr int vs_at(int r, int b) { return OFF_VS + (r >> 1) * (2 * NB) + 2 * b + (r & 1); }
};

inline int kv_unit_bytes(int head_dim, int fmt) { return 16 * head_dim + 32 * (head_dim / (fmt == MXQ_NVFP4 ? 16 : 32)); }

// Status codes of the key/value cache kernels in the device status word (first writer wins).
constexpr int kStatusKvSlot = 0x200;   // a slot at or behind num_pages * page_size
constexpr int kStatusKvPage = 0x201;   // a block-table entry outside the cache
constexpr int kStatusKvRows = 0x202;   // q_start outside q or falling, or more than max_q rows
constexpr int kStatusKvLen = 0x203;    // a length that the block table cannot hold

__device__ __forceinline__ void kv_status(int* status, int code) { atomicCAS(status, 0, code); }

}  // namespace mxq
