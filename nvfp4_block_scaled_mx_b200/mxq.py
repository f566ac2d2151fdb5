"""Thin ctypes binding of libmxq.so (the C ABI in include/mxq.h).

The raw functions keep the C names and arguments (pointers as ints, sizes, enums, a stream
handle).  The tensor helpers below only allocate outputs with torch and marshal arguments; every
step of the computation runs in the library's kernels.  There is no fallback: if the library is
missing or the device is not an sm_100 part, the calls raise.
"""
import ctypes
import functools
import os

import torch

MXFP4, NVFP4, MXFP8 = 0, 1, 2
EVEN, CEIL = 0, 1
OUT_BF16, OUT_FP32 = 0, 1
SF_ROWMAJOR, SF_SWIZZLED = 0, 1

FMT = {"mxfp4": MXFP4, "nvfp4": NVFP4, "mxfp8": MXFP8}
RULE = {"even": EVEN, "ceil": CEIL}

ERR_SHAPE = -2
ERR_TIMEOUT = -7

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmxq.so")

# name -> (restype, argtypes)
_P, _I64, _I, _SZ, _U64 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64
SIGNATURES = {
    "mxq_block_size": (_I, [_I]),
    "mxq_q_bytes": (_I, [_I64, _I64, _I, ctypes.POINTER(_SZ)]),
    "mxq_sf_bytes": (_I, [_I64, _I64, _I, _I, ctypes.POINTER(_SZ)]),
    "mxq_quantize": (_I, [_P, _I64, _I64, _I, _I, _P, _P, _P, _I, _P]),
    "mxq_quantize_running": (_I, [_P, _I64, _I64, _P, _P, _P, _P, _I, _P]),
    "mxq_fake_quantize": (_I, [_P, _I64, _I64, _I, _I, _P, _P, _P]),
    "mxq_swizzle_scales": (_I, [_P, _I64, _I64, _P, _P]),
    "mxq_global_scale": (_I, [_P, _I64, _P, _P, _P]),
    "mxq_amax": (_I, [_P, _I64, _P, _P]),
    "mxq_gemm": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _P, _P]),
    "mxq_gemm_w4a16": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _P, _P]),
    "mxq_linear_workspace_size": (_SZ, [_I64, _I64, _I]),
    "mxq_linear_kernel_count": (_I, [_I64, _I64, _I64, _I]),
    "mxq_linear": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _SZ, _P, _P]),
    "mxq_linear_noalloc": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _P, _P]),
    "mxq_kv_unit_bytes": (_I, [_I, _I, ctypes.POINTER(_SZ)]),
    "mxq_kv_append": (_I, [_P, _P, _I64, _I, _I, _I64, _I64, _I64, _I64, _P, _I, _I, _P, _P, _P, _I64, _I, _P]),
    "mxq_kv_read": (_I, [_P, _I64, _I, _I, _I, _I, _P, _I64, _P, _P, _P, _P, _P]),
    "mxq_kv_attention_workspace_size": (_SZ, [_I64, _I64, _I, _I, _I]),
    "mxq_kv_attention": (_I, [_P, _I64, _I64, _I64, _P, _I64, _I, _I, _I, _I, _I, _P, _I64, _I64, _P, _I64, _P, _I64,
                              ctypes.c_float, _I, _I64, _P, _P, _I, _P, _P, _P, _SZ, _P]),
    "mxq_kv_reserve_workspace_size": (_SZ, [_I64]),
    "mxq_kv_reserve": (_I, [_P, _P, _I64, _P, _I64, _I64, _I64, _P, _P, _I64, _I, _P, _I64, _I64, _I64, _P, _I64, _P, _P,
                            _SZ, _P]),
    "mxq_kv_fork": (_I, [_P, _P, _I64, _P, _I64, _I64, _I64, _P, _P, _I64, _I, _P, _P]),
    "mxq_kv_truncate": (_I, [_P, _P, _I64, _P, _I64, _I64, _I64, _P, _P, _I64, _I, _P, _P]),
    "mxq_kv_compact_workspace_size": (_SZ, [_I64]),
    "mxq_kv_compact": (_I, [_P, _I64, _I64, _I64, _P, _P, _I64, _I, _P, _I64, _I64, _I64, _P, _P, _SZ, _P]),
    "mxq_device_status": (_I, [ctypes.POINTER(_I), _I, _P]),
    "mxq_selftest_timeout": (_I, [_U64, _P]),
    "mxq_strerror": (ctypes.c_char_p, [_I]),
}

_lib = None


class MxqError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (where, lib().mxq_strerror(code).decode(), code))


class MxqBufferError(MxqError, ValueError):
    """A tensor handed to the binding does not fit the call (element type, rank or size); raised
    before anything reaches the library, with the shape error code."""

    def __init__(self, msg):
        self.code = ERR_SHAPE
        Exception.__init__(self, msg)


def lib():
    """Load libmxq.so (raises OSError if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise OSError("libmxq.so not built: run `python -m nvfp4_block_scaled_mx_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def _check(rc, where):
    if rc != 0:
        raise MxqError(rc, where)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("mxq works on CUDA tensors only (got a %s tensor)" % t.device)
    if not t.is_contiguous():
        raise ValueError("mxq needs contiguous tensors")
    return t.data_ptr()


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _fmt(f):
    return FMT[f] if isinstance(f, str) else int(f)


def _rule(r):
    return RULE[r] if isinstance(r, str) else int(r)


# ---------------------------------------------------------------- raw C entry points (same names)

def mxq_quantize(x, M, K, fmt, rule, global_scale, q_out, sf_out, layout, stream):
    return lib().mxq_quantize(x, M, K, fmt, rule, global_scale, q_out, sf_out, layout, stream)


def mxq_fake_quantize(x, M, K, fmt, rule, global_scale, y, stream):
    return lib().mxq_fake_quantize(x, M, K, fmt, rule, global_scale, y, stream)


def mxq_swizzle_scales(sf_rowmajor, rows, kblocks, sf_swizzled, stream):
    return lib().mxq_swizzle_scales(sf_rowmajor, rows, kblocks, sf_swizzled, stream)


def mxq_global_scale(x, n, g_out, amax_out, stream):
    return lib().mxq_global_scale(x, n, g_out, amax_out, stream)


def mxq_amax(x, n, amax_out, stream):
    return lib().mxq_amax(x, n, amax_out, stream)


def mxq_gemm(A_q, A_sf, B_q, B_sf, g_A, g_B, M, N, K, fmt, out_type, out, stream):
    return lib().mxq_gemm(A_q, A_sf, B_q, B_sf, g_A, g_B, M, N, K, fmt, out_type, out, stream)


def mxq_gemm_w4a16(A, W_q, W_sf, g_W, M, N, K, fmt, out_type, out, stream):
    return lib().mxq_gemm_w4a16(A, W_q, W_sf, g_W, M, N, K, fmt, out_type, out, stream)


def mxq_linear(x, W_q, W_sf, g_W, g_A, M, N, K, fmt, act_rule, out_type, workspace, ws_bytes, out, stream):
    return lib().mxq_linear(x, W_q, W_sf, g_W, g_A, M, N, K, fmt, act_rule, out_type, workspace, ws_bytes, out,
                            stream)


def mxq_linear_workspace_size(M, K, fmt):
    return lib().mxq_linear_workspace_size(M, K, fmt)


def linear_kernel_count(M, N, K, fmt):
    """Kernels one linear() call launches for this problem on the current device (1 or 2)."""
    n = lib().mxq_linear_kernel_count(M, N, K, _fmt(fmt))
    _check(n if n < 0 else 0, "mxq_linear_kernel_count")
    return n


def mxq_device_status(reset=True, stream=None):
    v = ctypes.c_int(0)
    _check(lib().mxq_device_status(ctypes.byref(v), 1 if reset else 0, _stream(stream)), "mxq_device_status")
    return v.value


def mxq_selftest_timeout(timeout_ns, stream=None):
    _check(lib().mxq_selftest_timeout(int(timeout_ns), _stream(stream)), "mxq_selftest_timeout")


# ---------------------------------------------------------------- tensor helpers

def block_size(fmt):
    return 16 if _fmt(fmt) == NVFP4 else 32


def q_shape(rows, K, fmt):
    return (rows, K if _fmt(fmt) == MXFP8 else K // 2)


def sf_bytes(rows, K, fmt, layout=SF_SWIZZLED):
    n = ctypes.c_size_t(0)
    _check(lib().mxq_sf_bytes(rows, K, _fmt(fmt), layout, ctypes.byref(n)), "mxq_sf_bytes")
    return n.value


def _q_bytes(rows, K, f):
    return rows * (K if f == MXFP8 else K // 2)


def _need(t, name, nbytes, dtype=None):
    """Host-side guard before a tensor's pointer crosses the C ABI, which sees no sizes: the kernels
    read or write `nbytes` through it, so a smaller buffer, or one of another element type where
    the element type matters, is refused here instead of being overrun on the device."""
    if t is None:
        return
    if dtype is not None and t.dtype != dtype:
        raise MxqBufferError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    have = t.numel() * t.element_size()
    if have < nbytes:
        raise MxqBufferError("%s holds %d bytes, the call needs %d" % (name, have, nbytes))


def _need_x(x, name="x"):
    if x.dim() != 2:
        raise MxqBufferError("%s must be a 2-D [M, K] tensor (got %d dims)" % (name, x.dim()))
    _need(x, name, 2 * x.numel(), torch.bfloat16)


def quantize(x, fmt, rule=EVEN, global_scale=None, layout=SF_SWIZZLED, q_out=None, sf_out=None, stream=None):
    """x [M, K] bf16 (CUDA) -> (q uint8 [M, K/2] or [M, K], sf uint8 flat (swizzled) or [M, K/bs])."""
    f, r = _fmt(fmt), _rule(rule)
    _need_x(x)
    M, K = x.shape
    if q_out is None:
        q_out = torch.empty(q_shape(M, K, f), dtype=torch.uint8, device=x.device)
    if sf_out is None:
        if layout == SF_SWIZZLED:
            sf_out = torch.empty(sf_bytes(M, K, f, layout), dtype=torch.uint8, device=x.device)
        else:
            sf_out = torch.empty((M, K // block_size(f)), dtype=torch.uint8, device=x.device)
    _need(q_out, "q_out", _q_bytes(M, K, f))
    _need(sf_out, "sf_out", sf_bytes(M, K, f, layout))
    _need(global_scale, "global_scale", 4, torch.float32)
    _check(mxq_quantize(_ptr(x), M, K, f, r, _ptr(global_scale), _ptr(q_out), _ptr(sf_out), layout,
                        _stream(stream)), "mxq_quantize")
    return q_out, sf_out


def quantize_running(x, amax_in, amax_out, layout=SF_SWIZZLED, q_out=None, sf_out=None, stream=None):
    """NVFP4 quantize of x with g = amax_in/2688; amax_out <- max(amax_in, max|x|)."""
    _need_x(x)
    M, K = x.shape
    if q_out is None:
        q_out = torch.empty(q_shape(M, K, NVFP4), dtype=torch.uint8, device=x.device)
    if sf_out is None:
        if layout == SF_SWIZZLED:
            sf_out = torch.empty(sf_bytes(M, K, NVFP4, layout), dtype=torch.uint8, device=x.device)
        else:
            sf_out = torch.empty((M, K // 16), dtype=torch.uint8, device=x.device)
    _need(q_out, "q_out", _q_bytes(M, K, NVFP4))
    _need(sf_out, "sf_out", sf_bytes(M, K, NVFP4, layout))
    _need(amax_in, "amax_in", 4, torch.float32)
    _need(amax_out, "amax_out", 4, torch.float32)
    _check(lib().mxq_quantize_running(_ptr(x), M, K, _ptr(amax_in), _ptr(amax_out), _ptr(q_out), _ptr(sf_out), layout,
                                      _stream(stream)), "mxq_quantize_running")
    return q_out, sf_out


def fake_quantize(x, fmt, rule=EVEN, global_scale=None, out=None, stream=None):
    """x [M, K] bf16 (CUDA) -> bf16 quantize-dequantize of x (out may be x for in-place)."""
    _need_x(x)
    M, K = x.shape
    if out is None:
        out = torch.empty_like(x)
    _need(out, "out", 2 * M * K, torch.bfloat16)
    _need(global_scale, "global_scale", 4, torch.float32)
    _check(mxq_fake_quantize(_ptr(x), M, K, _fmt(fmt), _rule(rule), _ptr(global_scale), _ptr(out), _stream(stream)),
           "mxq_fake_quantize")
    return out


def swizzle_scales(sf_rowmajor, out=None, stream=None):
    rows, kb = sf_rowmajor.shape
    n = ((rows + 127) // 128) * 128 * ((kb + 3) // 4) * 4
    if out is None:
        out = torch.empty(n, dtype=torch.uint8, device=sf_rowmajor.device)
    _need(sf_rowmajor, "sf_rowmajor", rows * kb, torch.uint8)
    _need(out, "out", n)
    _check(mxq_swizzle_scales(_ptr(sf_rowmajor), rows, kb, _ptr(out), _stream(stream)), "mxq_swizzle_scales")
    return out


def global_scale(x, stream=None):
    """NVFP4 decode-direction global scale g = amax / 2688 and amax, as device fp32[1] tensors."""
    _need(x, "x", 2 * x.numel(), torch.bfloat16)
    g = torch.empty(1, dtype=torch.float32, device=x.device)
    amax = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(mxq_global_scale(_ptr(x), x.numel(), _ptr(g), _ptr(amax), _stream(stream)), "mxq_global_scale")
    return g, amax


def amax(x, stream=None):
    """max |x| over the whole tensor, as a device fp32[1] tensor."""
    _need(x, "x", 2 * x.numel(), torch.bfloat16)
    out = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(mxq_amax(_ptr(x), x.numel(), _ptr(out), _stream(stream)), "mxq_amax")
    return out


def gemm(A_q, A_sf, B_q, B_sf, M, N, K, fmt, out_dtype=torch.bfloat16, g_A=None, g_B=None, out=None, stream=None):
    f = _fmt(fmt)
    ot = OUT_FP32 if out_dtype == torch.float32 else OUT_BF16
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A_q.device)
    _need(A_q, "A_q", _q_bytes(M, K, f))
    _need(B_q, "B_q", _q_bytes(N, K, f))
    _need(A_sf, "A_sf", sf_bytes(M, K, f))
    _need(B_sf, "B_sf", sf_bytes(N, K, f))
    _need(g_A, "g_A", 4, torch.float32)
    _need(g_B, "g_B", 4, torch.float32)
    _need(out, "out", M * N * (4 if ot == OUT_FP32 else 2), torch.float32 if ot == OUT_FP32 else torch.bfloat16)
    _check(mxq_gemm(_ptr(A_q), _ptr(A_sf), _ptr(B_q), _ptr(B_sf), _ptr(g_A), _ptr(g_B), M, N, K, f, ot, _ptr(out),
                    _stream(stream)), "mxq_gemm")
    return out


def gemm_w4a16(A, W_q, W_sf, N, fmt, g_W=None, out_dtype=torch.bfloat16, out=None, stream=None):
    """Weight-only GEMM: out = A dq(W)^T with A [M, K] bf16 and W pre-quantized (swizzled scales)."""
    f = _fmt(fmt)
    _need_x(A, "A")
    M, K = A.shape
    ot = OUT_FP32 if out_dtype == torch.float32 else OUT_BF16
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=A.device)
    if f == MXFP8:  # 4-bit weights only: the library rejects the format before any launch
        _check(mxq_gemm_w4a16(_ptr(A), _ptr(W_q), _ptr(W_sf), _ptr(g_W), M, N, K, f, ot, _ptr(out), _stream(stream)),
               "mxq_gemm_w4a16")
        return out
    _need(W_q, "W_q", _q_bytes(N, K, f))
    _need(W_sf, "W_sf", sf_bytes(N, K, f))
    _need(g_W, "g_W", 4, torch.float32)
    _need(out, "out", M * N * (4 if ot == OUT_FP32 else 2), torch.float32 if ot == OUT_FP32 else torch.bfloat16)
    _check(mxq_gemm_w4a16(_ptr(A), _ptr(W_q), _ptr(W_sf), _ptr(g_W), M, N, K, f, ot, _ptr(out), _stream(stream)),
           "mxq_gemm_w4a16")
    return out


def linear(x, W_q, W_sf, N, fmt, act_rule=CEIL, out_dtype=torch.bfloat16, g_W=None, g_A=None, workspace=None,
           out=None, stream=None):
    """Quantize x per token, then out = A_q W_q^T (W pre-quantized with swizzled scales)."""
    f = _fmt(fmt)
    _need_x(x)
    M, K = x.shape
    ws = mxq_linear_workspace_size(M, K, f)
    if workspace is None:
        workspace = torch.empty(ws, dtype=torch.uint8, device=x.device)
    ot = OUT_FP32 if out_dtype == torch.float32 else OUT_BF16
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _need(W_q, "W_q", _q_bytes(N, K, f))
    _need(W_sf, "W_sf", sf_bytes(N, K, f))
    _need(g_W, "g_W", 4, torch.float32)
    _need(g_A, "g_A", 4, torch.float32)
    _need(out, "out", M * N * (4 if ot == OUT_FP32 else 2), torch.float32 if ot == OUT_FP32 else torch.bfloat16)
    _check(mxq_linear(_ptr(x), _ptr(W_q), _ptr(W_sf), _ptr(g_W), _ptr(g_A), M, N, K, f, _rule(act_rule), ot,
                      _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(out), _stream(stream)),
           "mxq_linear")
    return out


# ---------------------------------------------------------------- 4-bit key/value cache
#
# These calls take a few microseconds on the device, so the checks in front of them are written to cost
# little: plain attribute reads, no device context unless the tensors lie on another device than the
# current one, and the current stream's handle straight from the runtime.

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_KV_UNIT = {(f, d): 16 * d + 32 * (d // b) for f, b in ((MXFP4, 32), (NVFP4, 16)) for d in (64, 128, 256)}


def kv_unit_bytes(head_dim, fmt):
    """Bytes of a unit of the cache: 16 tokens of one head, keys and values."""
    n = ctypes.c_size_t(0)
    _check(lib().mxq_kv_unit_bytes(head_dim, _fmt(fmt), ctypes.byref(n)), "mxq_kv_unit_bytes")
    return n.value


def kv_cache_shape(num_pages, kv_heads, head_dim, fmt, page_size, layers=None):
    """Shape of the uint8 tensor that holds one layer of the cache (or `layers` of them)."""
    if page_size % 16:
        raise MxqBufferError("page_size must be a multiple of 16 (got %d)" % page_size)
    shape = (num_pages, kv_heads, page_size // 16, kv_unit_bytes(head_dim, fmt))
    return shape if layers is None else (layers,) + shape


def _call(name, device, stream, *args):
    """The C call `name` on `device` (that of its tensors, whatever the current one is), on `stream` or the
    device's current stream."""
    index = device.index
    if index == torch._C._cuda_getDevice():
        rc = getattr(lib(), name)(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    else:
        if device.type != "cuda":
            raise ValueError("mxq works on CUDA tensors only (got %s tensors)" % device)
        with torch.cuda.device(device):
            rc = getattr(lib(), name)(*args, torch._C._cuda_getCurrentRawStream(index) if stream is None else stream.cuda_stream)
    if rc:
        raise MxqError(rc, name)


@functools.lru_cache(maxsize=1024)
def _attention_bytes(index, *sizes):
    """kv_attention_workspace on device `index` (a function of its arguments alone)."""
    with torch.cuda.device(index):
        return max(kv_attention_workspace(*sizes), 16)


def _empty(shape, dtype, device, stream):
    """Memory of the call's stream: what a freed block still waits for, or is given to next, is on that stream."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _at(t, name, dtype, n, device):
    """Pointer of a contiguous tensor of at least n elements of dtype on the call's device (None passes)."""
    if t is None:
        return None
    if t.dtype is dtype and t.device == device and t.numel() >= n and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise MxqBufferError("%s must be %s (got %s)" % (name, dtype, t.dtype))
    if t.device != device:
        raise MxqBufferError("%s is on %s, the call's other tensors on %s" % (name, t.device, device))
    if t.numel() < n:
        raise MxqBufferError("%s holds %d values, the call needs %d" % (name, t.numel(), n))
    raise MxqBufferError("%s must be contiguous" % name)


def _rows(t, name, device):
    """[tokens, heads, dim] bf16 whose last dimension is contiguous: pointer, token stride, head stride.  (The
    stride of a dimension of one entry is never used; torch leaves anything there.)"""
    n, h, d = t.shape
    s0, s1, s2 = t.stride()
    if t.dtype is not _BF16:
        raise MxqBufferError("%s must be torch.bfloat16 (got %s)" % (name, t.dtype))
    if s2 != 1 and d > 1:
        raise MxqBufferError("%s needs a contiguous last dimension" % name)
    if t.device != device:
        raise MxqBufferError("%s is on %s, the call's other tensors on %s" % (name, t.device, device))
    return t.data_ptr(), (s0 if n > 1 else 0), (s1 if h > 1 else 0)


def _kv_layer(cache, head_dim, f):
    """(pages, kv_heads, page_size) of one layer of the cache."""
    shape = cache.shape
    if cache.dtype is not _U8 or len(shape) != 4:
        raise MxqBufferError("cache must be uint8 [pages, kv_heads, page_size / 16, unit] (got %s %s)" %
                             (cache.dtype, tuple(shape)))
    pages, heads, units, unit = shape
    if unit != _KV_UNIT.get((f, head_dim), unit):  # (what the table does not hold, the library refuses)
        raise MxqBufferError("a unit of the cache holds %d bytes, heads of %d take %d" % (unit, head_dim, _KV_UNIT[f, head_dim]))
    return pages, heads, 16 * units


def kv_append(k, v, cache, slots, fmt, rule=CEIL, g_k=None, g_v=None, stream=None):
    """Quantize k, v [tokens, kv_heads, dim] bf16 (strided) into one layer of the cache at `slots` (int32,
    page * page_size + offset; negative: skipped)."""
    f, dev = _fmt(fmt), cache.device
    if k.dim() != 3 or k.shape != v.shape:
        raise MxqBufferError("k and v must be [tokens, kv_heads, dim] both (got %s, %s)" % (tuple(k.shape), tuple(v.shape)))
    T, H, D = k.shape
    pages, heads, page_size = _kv_layer(cache, D, f)
    if H != heads:
        raise MxqBufferError("k has %d heads, the cache %d" % (H, heads))
    kp, ks, kh = _rows(k, "k", dev)
    vp, vs, vh = _rows(v, "v", dev)
    _call("mxq_kv_append", dev, stream, kp, vp, T, H, D, ks, kh, vs, vh, _at(slots, "slots", _I32, T, dev), f, _rule(rule),
          _at(g_k, "g_k", _F32, 1, dev), _at(g_v, "g_v", _F32, 1, dev), _at(cache, "cache", _U8, 0, dev), pages, page_size)


def kv_read(cache, slots, fmt, head_dim, g_k=None, g_v=None, k_out=None, v_out=None, stream=None):
    """The tokens at `slots` of one layer of the cache as bf16 (k, v), each [tokens, kv_heads, head_dim]."""
    f, dev = _fmt(fmt), cache.device
    pages, H, page_size = _kv_layer(cache, head_dim, f)
    T = slots.numel()
    if k_out is None and v_out is None:  # one allocation
        k_out, v_out = _empty((2, T, H, head_dim), _BF16, dev, stream).unbind(0)
    elif k_out is None:
        k_out = _empty((T, H, head_dim), _BF16, dev, stream)
    elif v_out is None:
        v_out = _empty((T, H, head_dim), _BF16, dev, stream)
    n = T * H * head_dim
    _call("mxq_kv_read", dev, stream, _at(cache, "cache", _U8, 0, dev), pages, page_size, H, head_dim, f, _at(slots, "slots", _I32, T, dev), T,
          _at(g_k, "g_k", _F32, 1, dev), _at(g_v, "g_v", _F32, 1, dev), _at(k_out, "k_out", _BF16, n, dev),
          _at(v_out, "v_out", _BF16, n, dev))
    return k_out, v_out


def kv_attention_workspace(batch, max_q, heads, kv_heads, head_dim):
    """Workspace bytes of kv_attention on the current device."""
    return lib().mxq_kv_attention_workspace_size(batch, max_q, heads, kv_heads, head_dim)


def kv_attention(q, cache, block_table, kv_lens, fmt, q_start=None, max_q=None, scale=None, causal=True, window=0, g_k=None,
                 g_v=None, out_dtype=torch.bfloat16, out=None, lse=None, workspace=None, stream=None):
    """Attention of q [rows, heads, dim] bf16 (strided) over one layer of the cache: (out [rows, heads, dim],
    lse [rows, heads] fp32, natural logarithm).

    block_table int32 [batch, pages], kv_lens int32 [batch] (the query tokens included), q_start int32
    [batch + 1] (None: max_q rows a sequence, 1 by default).  With q_start, max_q is the most rows that any sequence
    may have; None takes all of q's, which is always right, but a batch of one or few rows each is faster with its own
    bound (kernel and workspace go by it).  scale: dim ** -0.5 by default.  Rows that see no token get zeros and
    -inf; rows of no sequence, and of one with more than max_q, are left as they were (what the call allocates
    itself holds anything there), the latter recorded in mxq_device_status."""
    f, dev = _fmt(fmt), q.device
    if q.dim() != 3 or block_table.dim() != 2:
        raise MxqBufferError("q must be [rows, heads, dim] and block_table [batch, pages] (got %s, %s)" %
                             (tuple(q.shape), tuple(block_table.shape)))
    rows, heads, D = q.shape
    pages, kv_heads, page_size = _kv_layer(cache, D, f)
    qp, qs, qh = _rows(q, "q", dev)
    batch, cols = block_table.shape
    if max_q is None:
        max_q = 1 if q_start is None else max(rows, 1)
    t0, t1 = block_table.stride()
    if (t1 != 1 and cols > 1) or block_table.dtype is not _I32 or block_table.device != dev:
        raise MxqBufferError("block_table must be torch.int32 [batch, pages] with contiguous rows, on the call's device")
    if out is None:
        out = _empty((rows, heads, D), out_dtype, dev, stream)
    dtype = out.dtype
    if dtype is not _F32 and dtype is not _BF16:
        raise MxqBufferError("out must be torch.bfloat16 or torch.float32 (got %s)" % dtype)
    if lse is None:
        lse = _empty((rows, heads), _F32, dev, stream)
    if workspace is None:
        size = _attention_bytes(dev.index, batch, max_q, heads, kv_heads, D) if q.is_cuda else 16
        workspace = _empty(size, _U8, dev, stream)
    _call("mxq_kv_attention", dev, stream, qp, rows, qs, qh, _at(cache, "cache", _U8, 0, dev), pages, page_size, heads, kv_heads, D, f,
          block_table.data_ptr(), t0 if batch > 1 else max(cols, 1), cols, _at(kv_lens, "kv_lens", _I32, batch, dev),
          batch, _at(q_start, "q_start", _I32, batch + 1, dev), max_q, D ** -0.5 if scale is None else scale, causal, window,
          _at(g_k, "g_k", _F32, 1, dev), _at(g_v, "g_v", _F32, 1, dev), dtype is _F32,
          _at(out, "out", dtype, rows * heads * D, dev), _at(lse, "lse", _F32, rows * heads, dev),
          _at(workspace, "workspace", workspace.dtype, 0, dev), workspace.numel() * workspace.element_size())
    return out, lse


def _pages_args(block_table, kv_lens, refs, info, page_size, stream):
    """Checks the page state; the arguments that all page calls share, and info."""
    dev = refs.device
    if block_table.dim() != 2 or not block_table.is_contiguous():
        raise MxqBufferError("block_table must be a contiguous [rows, pages] tensor")
    rows, cols = block_table.shape
    if info is None:
        info = _empty(2, _I32, dev, stream)
    return (_at(block_table, "block_table", _I32, 0, dev), rows, cols, cols, _at(kv_lens, "kv_lens", _I32, rows, dev),
            _at(refs, "refs", _I32, 1, dev), refs.numel(), page_size), info


def _kv_layers(cache, page_size, num_pages, dev):
    """Pointer, layers, layer stride and bytes of a page of a cache of one or more layers."""
    if cache.dtype is not _U8 or cache.dim() not in (4, 5):
        raise MxqBufferError("cache must be a contiguous uint8 [(layers,) pages, kv_heads, page_size / 16, unit] tensor")
    layers = cache.shape[0] if cache.dim() == 5 else 1
    pages, heads, units, unit = cache.shape[-4:]
    if pages < num_pages or 16 * units != page_size:
        raise MxqBufferError("the cache has %d pages of %d tokens, the call is for %d of %d" %
                             (pages, 16 * units, num_pages, page_size))
    return _at(cache, "cache", _U8, 0, dev), layers, pages * heads * units * unit, heads * units * unit


def kv_reserve(seqs, add, block_table, kv_lens, refs, cache, page_size, slots=None, info=None, workspace=None, stream=None):
    """Room for add[i] more tokens in row seqs[i] (int32 each); `cache` is [pages, ...] or [layers, pages, ...].
    slots receives the new tokens' slots, then -1.  Returns info (int32[2]: status, pages taken)."""
    state, info = _pages_args(block_table, kv_lens, refs, info, page_size, stream)
    n, dev = seqs.numel(), refs.device
    layers = _kv_layers(cache, page_size, refs.numel(), dev)
    if workspace is None:
        workspace = _empty(16 + 8 * n, _U8, dev, stream)
    _call("mxq_kv_reserve", dev, stream, _at(seqs, "seqs", _I32, n, dev), _at(add, "add", _I32, n, dev), n, *state, *layers,
          _at(slots, "slots", _I32, 0, dev), 0 if slots is None else slots.numel(), _at(info, "info", _I32, 2, dev),
          _at(workspace, "workspace", workspace.dtype, 0, dev), workspace.numel() * workspace.element_size())
    return info


def kv_fork(parents, children, block_table, kv_lens, refs, page_size, info=None, stream=None):
    """Empty row children[i] becomes a copy of row parents[i] that shares its pages.  Returns info."""
    state, info = _pages_args(block_table, kv_lens, refs, info, page_size, stream)
    n, dev = parents.numel(), refs.device
    _call("mxq_kv_fork", dev, stream, _at(parents, "parents", _I32, n, dev), _at(children, "children", _I32, n, dev), n,
          *state, _at(info, "info", _I32, 2, dev))
    return info


def kv_truncate(seqs, new_lens, block_table, kv_lens, refs, page_size, info=None, stream=None):
    """Cut row seqs[i] to new_lens[i] tokens (0 frees it).  Returns info."""
    state, info = _pages_args(block_table, kv_lens, refs, info, page_size, stream)
    n, dev = seqs.numel(), refs.device
    _call("mxq_kv_truncate", dev, stream, _at(seqs, "seqs", _I32, n, dev), _at(new_lens, "new_lens", _I32, n, dev), n, *state,
          _at(info, "info", _I32, 2, dev))
    return info


def kv_compact_workspace(num_pages):
    """Workspace bytes of kv_compact."""
    return lib().mxq_kv_compact_workspace_size(num_pages)


def kv_compact(block_table, kv_lens, refs, cache, page_size, info=None, workspace=None, stream=None):
    """Pack the pages in use to the front of the cache.  Returns info (int32[2]: 0, pages in use)."""
    state, info = _pages_args(block_table, kv_lens, refs, info, page_size, stream)
    dev = refs.device
    layers = _kv_layers(cache, page_size, refs.numel(), dev)
    if workspace is None:
        workspace = _empty(kv_compact_workspace(refs.numel()), _U8, dev, stream)
    _call("mxq_kv_compact", dev, stream, *state, *layers, _at(info, "info", _I32, 2, dev),
          _at(workspace, "workspace", workspace.dtype, 0, dev), workspace.numel() * workspace.element_size())
    return info
