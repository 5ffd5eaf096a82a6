"""Exact low-bit integer GEMM for AMD MI355X (gfx950) -- Python binding.

A thin ctypes layer over ``liblbgemm.so`` whose C ABI is declared in
``include/lb_gemm.h``.  The functions keep the C names and only marshal
arguments: they read shapes from the tensors, check dtypes, devices and
contiguity, and pass raw device pointers and torch's current HIP stream to the
library.  Every step of the computation runs in the library's HIP kernels;
there is no CPU or PyTorch fallback, and importing fails loudly when the
library has not been built.

Operand conventions (see the header): A is (M, K) row-major, B is given as its
(N, K) row-major rows (a column-major K x N matrix), C is (M, N) int32.  int4
operands are (rows, K/2) uint8 with the even k in the low nibble; 1-bit
operands are (rows, K/32) 32-bit words (torch.int32 or torch.uint32 bit
patterns) with element k in bit k % 32 of word k // 32.  Convolutions take an
NHWC image X (N, H, W, C), filters F (Co, Kh, Kw, C) and write Y (N, Ho, Wo,
Co) int32; int4 tensors hold C/2 bytes in the last dimension.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblbgemm.so")

LB_OK, LB_ERR_NULL, LB_ERR_SHAPE, LB_ERR_ALIGN, LB_ERR_VARIANT, LB_ERR_OVERFLOW, LB_ERR_HIP, \
    LB_ERR_WORKSPACE = range(8)
LB_S8, LB_S4, LB_B1 = 0, 1, 2
LB_BF16, LB_F16, LB_F32 = 0, 1, 2   # lb_ftype
LB_PLAN_LINEAR = 3   # lb_auto_plan's op code for the linear layer
LB_PLAN_SCALED = 5   # and for the scaled product
LB_AUTO = -1
LB_NUM_VARIANTS = 9
LB_DEFAULT_VARIANT = 7
K_ALIGN = {LB_S8: 16, LB_S4: 32, LB_B1: 128}
K_MAX = {LB_S8: 131071, LB_S4: 131071, LB_B1: 134217600}
# Longest 1-bit K one kernel pass covers, per matrix-instruction route (FP4, the
# default, sums in fp32, exact to 2^24; the int8 route, LB_B1_ROUTE=int8, sums 64
# per pair in int32); longer K runs as K bands (see the header).
B1_PASS_K = {"fp4": 1 << 24, "int8": 33554304}
KV4_PAGE_ALIGN = 16
KV4_HEAD_DIMS = (64, 128, 256)
CONV_C_ALIGN = {LB_S8: 16, LB_S4: 32}

# Exported symbols of include/lb_gemm.h (checked by the CPU tests).
EXPORTS = ("lb_gemm_s8", "lb_gemm_s4", "lb_gemm_b1", "lb_gemm_s8_linear", "lb_conv2d_s8",
           "lb_conv2d_s4", "lb_select_variant", "lb_status_string", "lb_variant_info",
           "lb_build_id", "lb_auto_plan", "lb_quant_rows_s8", "lb_gemm_s8_scaled", "lb_linear_w8a8",
           "lb_linear_w8a8_workspace", "lb_kv4_write", "lb_kv4_read", "lb_attn_kv4",
           "lb_attn_kv4_workspace")


class LbError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} (status {status})")


_lib = None


def load(path: str = LIB_PATH):
    """Load the library (once).  Raises if it has not been built, or if it was
    built from sources other than the ones in this tree (its lb_build_id()
    differs from the hash of csrc/ and include/)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} not found: build it with `python -m bit_integer_gemm_amd._build`")
    lib = ctypes.CDLL(path)
    lib.lb_build_id.argtypes = []
    lib.lb_build_id.restype = ctypes.c_char_p
    from . import _build
    built, want = lib.lb_build_id().decode(), _build.source_sha()
    if built != want:
        raise ImportError(f"{path} was built from sources {built}, the tree holds {want}: "
                          "rebuild with `python -m bit_integer_gemm_amd._build`")
    p, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    for name in ("lb_gemm_s8", "lb_gemm_s4", "lb_gemm_b1"):
        f = getattr(lib, name)
        f.argtypes = [p, p, p, i64, i64, i64, i32, p]
        f.restype = i32
    lib.lb_gemm_s8_linear.argtypes = [p, p, p, p, p, i64, i64, i64, i32, p]
    lib.lb_gemm_s8_linear.restype = i32
    for name in ("lb_conv2d_s8", "lb_conv2d_s4"):
        f = getattr(lib, name)
        f.argtypes = [p, p, p] + [i64] * 11 + [i32, p]
        f.restype = i32
    ip = ctypes.POINTER(ctypes.c_int)
    lib.lb_select_variant.argtypes = [i32, i64, i64, i64, i32, ip, ip]
    lib.lb_select_variant.restype = i32
    lib.lb_status_string.argtypes = [i32]
    lib.lb_status_string.restype = ctypes.c_char_p
    lib.lb_variant_info.argtypes = [i32, i32, ip, ip, ip, ip]
    lib.lb_variant_info.restype = i32
    lib.lb_auto_plan.argtypes = [i32, i64, i64, i64, i32, ip, ip, ip, ip]
    lib.lb_auto_plan.restype = i32
    lib.lb_quant_rows_s8.argtypes = [p, i64, p, p, i64, i64, i32, p]
    lib.lb_gemm_s8_scaled.argtypes = [p] * 6 + [i64] * 3 + [i32, p]
    lib.lb_linear_w8a8.argtypes = [p, i64, p, p, p, p, i64, i64, i64, i32, p, i64, p]
    lib.lb_linear_w8a8_workspace.argtypes = [i64] * 3
    lib.lb_linear_w8a8_workspace.restype = i64
    lib.lb_kv4_write.argtypes = [p, p, i64, i64] + [p] * 5 + [i64] * 5 + [i32, p]
    lib.lb_kv4_read.argtypes = [p] * 7 + [i64] * 5 + [i32, p]
    lib.lb_attn_kv4.argtypes = ([p, i64, p, p, p, p, p, i64, i64, p, p, p, i64, p] + [i64] * 9 +
                                [ctypes.c_float, i64, i32, i32, p, i64, p])
    lib.lb_attn_kv4_workspace.argtypes = [i64] * 8 + [i32]
    lib.lb_attn_kv4_workspace.restype = i64
    for name in ("lb_quant_rows_s8", "lb_gemm_s8_scaled", "lb_linear_w8a8", "lb_kv4_write", "lb_kv4_read",
                 "lb_attn_kv4"):
        getattr(lib, name).restype = i32
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().lb_status_string(status).decode()


def build_id() -> str:
    """Source hash stamped into the loaded library."""
    return load().lb_build_id().decode()


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

def _stream_handle(stream, device_index):
    import torch
    if stream is None:
        # torch's current stream on the operands' device (raw hipStream_t)
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(device_index))
    return ctypes.c_void_p(int(getattr(stream, "cuda_stream", stream)))


def _check(t, dtypes, shape, what):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be on a GPU (got {t.device})")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: dtype {t.dtype} not in {dtypes}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)} != {tuple(shape)}")


def _same_device(*ts):
    d = ts[0].get_device()
    for t in ts[1:]:
        if t.get_device() != d:
            raise ValueError("all operands must be on the same GPU")
    return d


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _raise(st, where):
    if st != LB_OK:
        raise LbError(st, where)


# ---------------------------------------------------------------------------
# the C ABI, one function each
# ---------------------------------------------------------------------------

def lb_gemm_s8(A, B, C, variant: int = LB_AUTO, stream=None) -> None:
    """C (M, N) int32 = A (M, K) int8 x B, B given as (N, K) int8 rows."""
    import torch
    M, K = A.shape
    N = B.shape[0]
    _check(A, (torch.int8,), (M, K), "A")
    _check(B, (torch.int8,), (N, K), "B")
    _check(C, (torch.int32,), (M, N), "C")
    _raise(load().lb_gemm_s8(_ptr(A), _ptr(B), _ptr(C), M, N, K, variant,
                             _stream_handle(stream, _same_device(A, B, C))), "lb_gemm_s8")


def lb_gemm_s4(A, B, C, variant: int = LB_AUTO, stream=None) -> None:
    """C (M, N) int32 = A x B for packed int4: A (M, K/2) uint8, B (N, K/2) uint8."""
    import torch
    M, Kh = A.shape
    N = B.shape[0]
    _check(A, (torch.uint8,), (M, Kh), "A")
    _check(B, (torch.uint8,), (N, Kh), "B")
    _check(C, (torch.int32,), (M, N), "C")
    _raise(load().lb_gemm_s4(_ptr(A), _ptr(B), _ptr(C), M, N, 2 * Kh, variant,
                             _stream_handle(stream, _same_device(A, B, C))), "lb_gemm_s4")


def lb_gemm_b1(A, B, C, variant: int = LB_AUTO, stream=None) -> None:
    """C (M, N) int32 = popcount(A AND B) over K bits: A (M, K/32), B (N, K/32) words."""
    import torch
    words = (torch.int32, torch.uint32)
    M, Kw = A.shape
    N = B.shape[0]
    _check(A, words, (M, Kw), "A")
    _check(B, words, (N, Kw), "B")
    _check(C, (torch.int32,), (M, N), "C")
    _raise(load().lb_gemm_b1(_ptr(A), _ptr(B), _ptr(C), M, N, 32 * Kw, variant,
                             _stream_handle(stream, _same_device(A, B, C))), "lb_gemm_b1")


def lb_gemm_s8_linear(X, W, sx, sw, out, variant: int = LB_AUTO, stream=None) -> None:
    """out (M, N) fp32 = (X (M, K) int8 x W (N, K) int8) * sx[m] * sw[n]."""
    import torch
    M, K = X.shape
    N = W.shape[0]
    _check(X, (torch.int8,), (M, K), "X")
    _check(W, (torch.int8,), (N, K), "W")
    _check(sx, (torch.float32,), (M,), "sx")
    _check(sw, (torch.float32,), (N,), "sw")
    _check(out, (torch.float32,), (M, N), "out")
    _raise(load().lb_gemm_s8_linear(_ptr(X), _ptr(W), _ptr(sx), _ptr(sw), _ptr(out), M, N, K, variant,
                                    _stream_handle(stream, _same_device(X, W, sx, sw, out))),
           "lb_gemm_s8_linear")


def conv_out_dims(H: int, W: int, Kh: int, Kw: int, stride=(1, 1), pad=(0, 0)):
    """(Ho, Wo) of a convolution (the formula in the header)."""
    return (H + 2 * pad[0] - Kh) // stride[0] + 1, (W + 2 * pad[1] - Kw) // stride[1] + 1


def _conv(name, dtype, X, F, Y, stride, pad, variant, stream, cdiv):
    N, H, W, cl = X.shape
    Co, Kh, Kw, cl2 = F.shape
    C = cl * cdiv
    Ho, Wo = conv_out_dims(H, W, Kh, Kw, stride, pad)
    _check(X, (dtype,), (N, H, W, cl), "X")
    _check(F, (dtype,), (Co, Kh, Kw, cl), "F")
    import torch
    _check(Y, (torch.int32,), (N, Ho, Wo, Co), "Y")
    fn = getattr(load(), name)
    _raise(fn(_ptr(X), _ptr(F), _ptr(Y), N, H, W, C, Co, Kh, Kw, stride[0], stride[1], pad[0], pad[1],
              variant, _stream_handle(stream, _same_device(X, F, Y))), name)


def lb_conv2d_s8(X, F, Y, stride=(1, 1), pad=(0, 0), variant: int = LB_AUTO, stream=None) -> None:
    """Y (N, Ho, Wo, Co) int32 = convolution of X (N, H, W, C) int8 with F (Co, Kh, Kw, C) int8."""
    import torch
    _conv("lb_conv2d_s8", torch.int8, X, F, Y, tuple(stride), tuple(pad), variant, stream, 1)


def lb_conv2d_s4(X, F, Y, stride=(1, 1), pad=(0, 0), variant: int = LB_AUTO, stream=None) -> None:
    """As lb_conv2d_s8 for packed int4: X (N, H, W, C/2) uint8, F (Co, Kh, Kw, C/2) uint8."""
    import torch
    _conv("lb_conv2d_s4", torch.uint8, X, F, Y, tuple(stride), tuple(pad), variant, stream, 2)


def lb_select_variant(dtype: int, M: int, N: int, K: int, cu_count: int = 0):
    """(best, second) variant indices for a shape; cu_count <= 0 asks the device."""
    best, second = ctypes.c_int(-1), ctypes.c_int(-1)
    _raise(load().lb_select_variant(dtype, M, N, K, cu_count, ctypes.byref(best), ctypes.byref(second)),
           "lb_select_variant")
    return best.value, second.value


def lb_variant_info(dtype: int, variant: int) -> dict:
    """Workgroup tile (rows, columns, K elements per stage) and stage count of a variant."""
    vals = [ctypes.c_int(0) for _ in range(4)]
    _raise(load().lb_variant_info(dtype, variant, *[ctypes.byref(v) for v in vals]), "lb_variant_info")
    return dict(zip(("tile_m", "tile_n", "tile_k", "stages"), (v.value for v in vals)))


def lb_auto_plan(op: int, M: int, N: int, K: int, cu_count: int = 0) -> dict:
    """What an LB_AUTO call makes for a shape: the number of launches, the first
    launch's workgroup tile and its K bands.  op: LB_S8, LB_S4, LB_B1,
    LB_PLAN_LINEAR or LB_PLAN_SCALED; cu_count <= 0 plans for the current device."""
    vals = [ctypes.c_int(0) for _ in range(4)]
    _raise(load().lb_auto_plan(op, M, N, K, cu_count, *[ctypes.byref(v) for v in vals]), "lb_auto_plan")
    return dict(zip(("launches", "tile_m", "tile_n", "k_bands"), (v.value for v in vals)))


def ops(dtype: int, M: int, N: int, K: int) -> int:
    """Operation count used for TOPS: 2*M*N*K (K in elements, or bits for 1-bit)."""
    return 2 * M * N * K


# ---------------------------------------------------------------------------
# serving operators: an int8 linear layer on floating activations, a paged cache
# in 4 bits and attention over it
# ---------------------------------------------------------------------------

# These run once per layer and token, where the host's time counts: one pass over the
# operands' attributes, and words only for an operand that is refused.

class _Torch:
    """torch and what the checks below take from it, looked up at the first call."""

    def __init__(self):
        import torch
        self.torch = torch
        self.i8, self.u8, self.i32, self.i64, self.f32 = (torch.int8, torch.uint8, torch.int32, torch.int64,
                                                          torch.float32)
        self.any = {torch.bfloat16: LB_BF16, torch.float16: LB_F16, torch.float32: LB_F32}
        self.short = {torch.bfloat16: LB_BF16, torch.float16: LB_F16}
        self.current_stream = torch._C._cuda_getCurrentRawStream


_t = None


def _torch():
    global _t
    if _t is None:
        _t = _Torch()
    return _t


def _refuse(t, what, dtype, shape, device, dense=True):
    """Raises for an operand that is not a GPU tensor of this type, shape and device."""
    if t.get_device() < 0:
        raise ValueError(f"{what} must be on a GPU (got {t.device})")
    if t.dtype != dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if t.shape != tuple(shape):
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.get_device() != device:
        raise ValueError(f"{what} is on another GPU")
    raise ValueError(f"{what}: strides {t.stride()}; " +
                     ("it must be contiguous" if dense else "only the first dimension may be strided"))


def _dense(t, what, dtype, shape, device):
    """Address of a contiguous tensor of this type, shape and GPU."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device or device < 0:
        _refuse(t, what, dtype, shape, device)
    return t.data_ptr()


def _rows(t, what, dtype, shape, device, row):
    """(address, elements between rows) of a tensor whose rows of `row` elements are dense, `row` the product
    of all dimensions but the first."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != device or device < 0:
        _refuse(t, what, dtype, shape, device)
    if t.is_contiguous():
        return t.data_ptr(), row
    st, dense = t.stride(), 1
    for d in range(len(st) - 1, 0, -1):
        if st[d] != dense and shape[d] != 1:
            _refuse(t, what, dtype, shape, device, dense=False)
        dense *= shape[d]
    return t.data_ptr(), st[0] if shape[0] > 1 else row


def _ftype(table, t, what):
    f = table.get(t.dtype)
    if f is None:
        raise TypeError(f"{what}: dtype {t.dtype} not in {tuple(table)}")
    return f


def _on(T, stream, device):
    if stream is None:
        return T.current_stream(device)
    return int(getattr(stream, "cuda_stream", stream))


def _scratch(T, workspace, needed, device, stream, what):
    """The workspace tensor: the caller's, or one from torch's allocator (then ordered on torch's current
    stream, so not with a stream argument), or None where none is needed."""
    if workspace is not None:
        if not workspace.is_contiguous() or workspace.get_device() != device:
            raise ValueError(f"{what}: the workspace must be contiguous and on the operands' GPU")
        return workspace
    if needed == 0:
        return None
    if stream is not None:
        raise ValueError(f"{what}: a call on a stream of its own needs a workspace of {needed} bytes")
    return T.torch.empty(needed, dtype=T.u8, device=f"cuda:{device}")


def lb_quant_rows_s8(X, Q, sx, stream=None) -> None:
    """Rows of X (M, K) bf16, fp16 or fp32 (rows may be strided) quantised to Q (M, K) int8 with a scale
    each, sx (M,) fp32 = largest magnitude / 127."""
    T = _torch()
    M, K = X.shape
    dev = X.get_device()
    f = _ftype(T.any, X, "X")
    x, ldx = _rows(X, "X", X.dtype, (M, K), dev, K)
    st = load().lb_quant_rows_s8(x, ldx, _dense(Q, "Q", T.i8, (M, K), dev), _dense(sx, "sx", T.f32, (M,), dev),
                                 M, K, f, _on(T, stream, dev))
    _raise(st, "lb_quant_rows_s8")


def lb_gemm_s8_scaled(X, W, sx, sw, out, bias=None, stream=None) -> None:
    """out (M, N) bf16, fp16 or fp32 = (X (M, K) int8 x W (N, K) int8) * sx[m] * sw[n] + bias[n]; bias (N,)
    of out's type or None."""
    T = _torch()
    M, K = X.shape
    N = W.shape[0]
    dev, dt = X.get_device(), out.dtype
    f = _ftype(T.any, out, "out")
    st = load().lb_gemm_s8_scaled(
        _dense(X, "X", T.i8, (M, K), dev), _dense(W, "W", T.i8, (N, K), dev), _dense(sx, "sx", T.f32, (M,), dev),
        _dense(sw, "sw", T.f32, (N,), dev), None if bias is None else _dense(bias, "bias", dt, (N,), dev),
        _dense(out, "out", dt, (M, N), dev), M, N, K, f, _on(T, stream, dev))
    _raise(st, "lb_gemm_s8_scaled")


def lb_linear_w8a8_workspace(M: int, K: int, N: int) -> int:
    """Workspace bytes of lb_linear_w8a8 for X (M, K) and W (N, K)."""
    return load().lb_linear_w8a8_workspace(M, K, N)


def lb_linear_w8a8(X, W, sw, out, bias=None, workspace=None, stream=None) -> None:
    """out (M, N) = (round(127 X / amax) x W (N, K) int8) * (amax / 127) * sw[n] + bias[n], amax the largest
    magnitude of each row of X (M, K).  X (rows may be strided), bias and out share a type: bf16, fp16 or
    fp32.  workspace: a GPU tensor of at least lb_linear_w8a8_workspace(M, K, N) bytes, or None for one
    from torch's allocator."""
    T = _torch()
    lib = load()
    M, K = X.shape
    N = W.shape[0]
    dev, dt = X.get_device(), X.dtype
    f = _ftype(T.any, X, "X")
    x, ldx = _rows(X, "X", dt, (M, K), dev, K)
    w = _dense(W, "W", T.i8, (N, K), dev)
    s = _dense(sw, "sw", T.f32, (N,), dev)
    o = _dense(out, "out", dt, (M, N), dev)
    b = None if bias is None else _dense(bias, "bias", dt, (N,), dev)
    ws = _scratch(T, workspace, 0 if workspace is not None else lib.lb_linear_w8a8_workspace(M, K, N), dev, stream,
                  "lb_linear_w8a8")
    st = lib.lb_linear_w8a8(x, ldx, w, s, b, o, M, N, K, f, None if ws is None else ws.data_ptr(),
                            0 if ws is None else ws.nbytes, _on(T, stream, dev))
    _raise(st, "lb_linear_w8a8")


def _kv4_cache(T, Kc, Vc, Kp, Vp, heads, D, dtype, dev):
    """(pages, page, addresses) of the four tensors of a cache."""
    if Kc.dim() != 4:
        raise ValueError(f"Kc: expected (pages, heads, page, D/2), got {tuple(Kc.shape)}")
    shape = Kc.shape
    pages, h, page, half = shape
    if h != heads or 2 * half != D:
        raise ValueError(f"Kc: shape {tuple(shape)} does not fit {heads} heads of {D}")
    prm = (pages, h, page, 2)
    return pages, page, (_dense(Kc, "Kc", T.u8, shape, dev), _dense(Vc, "Vc", T.u8, shape, dev),
                         _dense(Kp, "Kp", dtype, prm, dev), _dense(Vp, "Vp", dtype, prm, dev))


def lb_kv4_write(K, V, slots, Kc, Vc, Kp, Vp, stream=None) -> None:
    """Keys and values of new tokens, K and V (T, heads, D) bf16 or fp16 (tokens may be strided), quantised
    to 4 bits into their slots (T,) int64 of the paged cache: Kc, Vc (pages, heads, page, D/2) uint8 and
    Kp, Vp (pages, heads, page, 2), scale and minimum of each vector in K's type.  Slots outside the cache
    (-1) are skipped."""
    T = _torch()
    shape = n, H, D = K.shape
    dev, dt = K.get_device(), K.dtype
    f = _ftype(T.short, K, "K")
    k, ldk = _rows(K, "K", dt, shape, dev, H * D)
    v, ldv = _rows(V, "V", dt, shape, dev, H * D)
    pages, page, cache = _kv4_cache(T, Kc, Vc, Kp, Vp, H, D, dt, dev)
    st = load().lb_kv4_write(k, v, ldk, ldv, _dense(slots, "slots", T.i64, (n,), dev), *cache, n, H, D, pages,
                             page, f, _on(T, stream, dev))
    _raise(st, "lb_kv4_write")


def lb_kv4_read(Kc, Vc, Kp, Vp, slots, K, V, stream=None) -> None:
    """Keys and values of slots (T,) int64 of the cache into K and V (T, heads, D); slots outside it read
    as zeros."""
    T = _torch()
    shape = n, H, D = K.shape
    dev, dt = K.get_device(), K.dtype
    f = _ftype(T.short, K, "K")
    pages, page, cache = _kv4_cache(T, Kc, Vc, Kp, Vp, H, D, dt, dev)
    st = load().lb_kv4_read(*cache, _dense(slots, "slots", T.i64, (n,), dev), _dense(K, "K", dt, shape, dev),
                            _dense(V, "V", dt, shape, dev), n, H, D, pages, page, f, _on(T, stream, dev))
    _raise(st, "lb_kv4_read")


def lb_attn_kv4_workspace(B: int, total_q: int, max_q: int, Hq: int, Hkv: int, D: int, max_len: int,
                          window: int = 0, cu_count: int = 0) -> int:
    """Workspace bytes with which lb_attn_kv4 splits the keys as it likes."""
    return load().lb_attn_kv4_workspace(B, total_q, max_q, Hq, Hkv, D, max_len, window, cu_count)


def lb_attn_kv4(Q, Kc, Vc, Kp, Vp, table, q_off, lens, out, lse=None, max_q=None, max_len=None, scale=None,
                window: int = 0, causal: bool = True, workspace=None, stream=None) -> None:
    """out (total_q, Hq, D) = attention of the last queries of each of B sequences over its pages.

    Q (total_q, Hq, D): rows q_off[b] .. q_off[b+1] - 1 (q_off (B + 1,) int32) are the last queries of
    sequence b, whose lens[b] (int32) keys lie in the pages table[b] (B, width) int32 names.  lse
    (total_q, Hq) fp32 receives the log of each row's sum, if given.  max_q: at least the most queries of a
    sequence; it chooses the kernel, so pass 1 for single tokens and the draft's length for drafts.  The
    default, total_q, is right for any batch but meant for one prompt: 64 single tokens take four times as
    long with it (256 against 69 us at up to 8191 keys).  max_len: about the longest sequence, for the
    planning (default: the table's width).  scale defaults to D ** -0.5; window > 0 keeps the last window keys.  A query that sees
    nothing gets zeros.  workspace: as for lb_linear_w8a8; a smaller one splits the keys less."""
    T = _torch()
    lib = load()
    shape = total, Hq, D = Q.shape
    dev, dt = Q.get_device(), Q.dtype
    f = _ftype(T.short, Q, "Q")
    rows = B, width = table.shape
    Hkv = Kc.shape[1]
    q, ldq = _rows(Q, "Q", dt, shape, dev, Hq * D)
    o, ldo = _rows(out, "out", dt, shape, dev, Hq * D)
    t, ldt = _rows(table, "table", T.i32, rows, dev, width)
    pages, page, cache = _kv4_cache(T, Kc, Vc, Kp, Vp, Hkv, D, dt, dev)
    if max_q is None:
        max_q = total
    if max_len is None:
        max_len = width * page
    ws = _scratch(T, workspace, 0 if workspace is not None else
                  lib.lb_attn_kv4_workspace(B, total, max_q, Hq, Hkv, D, max_len, window, 0), dev, stream, "lb_attn_kv4")
    st = lib.lb_attn_kv4(q, ldq, *cache, t, ldt, width, _dense(q_off, "q_off", T.i32, (B + 1,), dev),
                         _dense(lens, "lens", T.i32, (B,), dev), o, ldo,
                         None if lse is None else _dense(lse, "lse", T.f32, (total, Hq), dev), B, total, max_q, Hq,
                         Hkv, D, pages, page, max_len, D ** -0.5 if scale is None else scale, window, int(causal), f,
                         None if ws is None else ws.data_ptr(), 0 if ws is None else ws.nbytes, _on(T, stream, dev))
    _raise(st, "lb_attn_kv4")
