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
    launch's workgroup tile and its K bands.  op: LB_S8, LB_S4, LB_B1 or
    LB_PLAN_LINEAR; cu_count <= 0 plans for the current device."""
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

_FTYPES = {}


def _ftype(t, what, short=False):
    if not _FTYPES:
        import torch
        _FTYPES.update({torch.bfloat16: LB_BF16, torch.float16: LB_F16, torch.float32: LB_F32})
    f = _FTYPES.get(t.dtype)
    if f is None or (short and f == LB_F32):
        raise TypeError(f"{what}: dtype {t.dtype} is not a {'16-bit ' if short else ''}floating type of the library")
    return f


def _rows(t, dtype, shape, what):
    """A GPU tensor whose last dimensions are dense and whose first has any stride; returns that stride."""
    if t.dtype != dtype or not t.is_cuda or t.shape != shape:
        raise ValueError(f"{what}: expected a {dtype} GPU tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    st = t.stride()
    dense = 1
    for d in range(len(st) - 1, 0, -1):
        if st[d] != dense and shape[d] != 1:
            raise ValueError(f"{what}: only the first dimension may be strided (strides {st})")
        dense *= shape[d]
    return st[0] if shape[0] > 1 else max(st[0], dense)


def _dense(t, dtype, shape, what):
    if t.dtype != dtype or not t.is_cuda or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous {dtype} GPU tensor of shape {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)} with strides {t.stride()} on {t.device}")


def _raw_stream(stream, device):
    import torch
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    return int(getattr(stream, "cuda_stream", stream))


def _scratch(workspace, needed, t, stream, what):
    """(address, bytes) of a caller's workspace, or of one from torch's allocator
    (then ordered on torch's current stream, so not with a stream argument), and
    the tensor that keeps it."""
    import torch
    if workspace is None:
        if needed == 0:
            return None, 0, None
        if stream is not None:
            raise ValueError(f"{what}: a call on a stream of its own needs a workspace of {needed} bytes")
        workspace = torch.empty(needed, dtype=torch.uint8, device=t.device)
    elif not workspace.is_contiguous() or workspace.get_device() != t.get_device():
        raise ValueError(f"{what}: the workspace must be contiguous and on the operands' GPU")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def lb_quant_rows_s8(X, Q, sx, stream=None) -> None:
    """Rows of X (M, K) bf16, fp16 or fp32 (rows may be strided) quantised to Q (M, K) int8 with a scale
    each, sx (M,) fp32 = largest magnitude / 127."""
    import torch
    M, K = X.shape
    ldx = _rows(X, X.dtype, (M, K), "X")
    _dense(Q, torch.int8, (M, K), "Q")
    _dense(sx, torch.float32, (M,), "sx")
    f = _ftype(X, "X")
    dev = _same_device(X, Q, sx)
    _raise(load().lb_quant_rows_s8(X.data_ptr(), ldx, Q.data_ptr(), sx.data_ptr(), M, K, f,
                                   _raw_stream(stream, dev)), "lb_quant_rows_s8")


def lb_gemm_s8_scaled(X, W, sx, sw, out, bias=None, stream=None) -> None:
    """out (M, N) bf16, fp16 or fp32 = (X (M, K) int8 x W (N, K) int8) * sx[m] * sw[n] + bias[n]; bias (N,)
    of out's type or None."""
    import torch
    M, K = X.shape
    N = W.shape[0]
    _dense(X, torch.int8, (M, K), "X")
    _dense(W, torch.int8, (N, K), "W")
    _dense(sx, torch.float32, (M,), "sx")
    _dense(sw, torch.float32, (N,), "sw")
    _dense(out, out.dtype, (M, N), "out")
    f = _ftype(out, "out")
    dev = _same_device(X, W, sx, sw, out)
    if bias is not None:
        _dense(bias, out.dtype, (N,), "bias")
        _same_device(bias, out)
    _raise(load().lb_gemm_s8_scaled(X.data_ptr(), W.data_ptr(), sx.data_ptr(), sw.data_ptr(),
                                    None if bias is None else bias.data_ptr(), out.data_ptr(), M, N, K, f,
                                    _raw_stream(stream, dev)), "lb_gemm_s8_scaled")


def lb_linear_w8a8_workspace(M: int, K: int, N: int) -> int:
    """Workspace bytes of lb_linear_w8a8 for X (M, K) and W (N, K)."""
    return load().lb_linear_w8a8_workspace(M, K, N)


def lb_linear_w8a8(X, W, sw, out, bias=None, workspace=None, stream=None) -> None:
    """out (M, N) = (round(127 X / amax) x W (N, K) int8) * (amax / 127) * sw[n] + bias[n], amax the largest
    magnitude of each row of X (M, K).  X (rows may be strided), bias and out share a type: bf16, fp16 or
    fp32.  workspace: a GPU tensor of at least lb_linear_w8a8_workspace(M, K, N) bytes, or None for one
    from torch's allocator."""
    import torch
    M, K = X.shape
    N = W.shape[0]
    ldx = _rows(X, X.dtype, (M, K), "X")
    _dense(W, torch.int8, (N, K), "W")
    _dense(sw, torch.float32, (N,), "sw")
    _dense(out, X.dtype, (M, N), "out")
    f = _ftype(X, "X")
    dev = _same_device(X, W, sw, out)
    if bias is not None:
        _dense(bias, X.dtype, (N,), "bias")
        _same_device(bias, out)
    lib = load()
    need = 0 if workspace is not None else lib.lb_linear_w8a8_workspace(M, K, N)
    ws, size, kept = _scratch(workspace, need, X, stream, "lb_linear_w8a8")
    _raise(lib.lb_linear_w8a8(X.data_ptr(), ldx, W.data_ptr(), sw.data_ptr(),
                              None if bias is None else bias.data_ptr(), out.data_ptr(), M, N, K, f, ws, size,
                              _raw_stream(stream, dev)), "lb_linear_w8a8")


def _kv4_cache(Kc, Vc, Kp, Vp, heads, D, like):
    """Checks the four tensors of a cache; returns (pages, page)."""
    import torch
    if Kc.dim() != 4:
        raise ValueError(f"Kc: expected (pages, heads, page, D/2), got {tuple(Kc.shape)}")
    pages, h, page, half = Kc.shape
    if h != heads or 2 * half != D:
        raise ValueError(f"Kc: shape {tuple(Kc.shape)} does not fit {heads} heads of {D}")
    _dense(Kc, torch.uint8, (pages, heads, page, half), "Kc")
    _dense(Vc, torch.uint8, (pages, heads, page, half), "Vc")
    _dense(Kp, like.dtype, (pages, heads, page, 2), "Kp")
    _dense(Vp, like.dtype, (pages, heads, page, 2), "Vp")
    return pages, page


def lb_kv4_write(K, V, slots, Kc, Vc, Kp, Vp, stream=None) -> None:
    """Keys and values of new tokens, K and V (T, heads, D) bf16 or fp16 (tokens may be strided), quantised
    to 4 bits into their slots (T,) int64 of the paged cache: Kc, Vc (pages, heads, page, D/2) uint8 and
    Kp, Vp (pages, heads, page, 2), scale and minimum of each vector in K's type.  Slots outside the cache
    (-1) are skipped."""
    import torch
    T, H, D = K.shape
    ldk = _rows(K, K.dtype, (T, H, D), "K")
    ldv = _rows(V, K.dtype, (T, H, D), "V")
    _dense(slots, torch.int64, (T,), "slots")
    f = _ftype(K, "K", short=True)
    pages, page = _kv4_cache(Kc, Vc, Kp, Vp, H, D, K)
    dev = _same_device(K, V, slots, Kc, Vc, Kp, Vp)
    _raise(load().lb_kv4_write(K.data_ptr(), V.data_ptr(), ldk, ldv, slots.data_ptr(), Kc.data_ptr(),
                               Vc.data_ptr(), Kp.data_ptr(), Vp.data_ptr(), T, H, D, pages, page, f,
                               _raw_stream(stream, dev)), "lb_kv4_write")


def lb_kv4_read(Kc, Vc, Kp, Vp, slots, K, V, stream=None) -> None:
    """Keys and values of slots (T,) int64 of the cache into K and V (T, heads, D); slots outside it read
    as zeros."""
    import torch
    T, H, D = K.shape
    _dense(K, K.dtype, (T, H, D), "K")
    _dense(V, K.dtype, (T, H, D), "V")
    _dense(slots, torch.int64, (T,), "slots")
    f = _ftype(K, "K", short=True)
    pages, page = _kv4_cache(Kc, Vc, Kp, Vp, H, D, K)
    dev = _same_device(K, V, slots, Kc, Vc, Kp, Vp)
    _raise(load().lb_kv4_read(Kc.data_ptr(), Vc.data_ptr(), Kp.data_ptr(), Vp.data_ptr(), slots.data_ptr(),
                              K.data_ptr(), V.data_ptr(), T, H, D, pages, page, f, _raw_stream(stream, dev)),
           "lb_kv4_read")


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
    sequence (default: total_q); max_len: about the longest sequence, for the planning (default: the
    table's width).  scale defaults to D ** -0.5; window > 0 keeps the last window keys.  A query that sees
    nothing gets zeros.  workspace: as for lb_linear_w8a8; a smaller one makes fewer key ranges."""
    import torch
    total, Hq, D = Q.shape
    B, width = table.shape
    Hkv = Kc.shape[1] if Kc.dim() == 4 else 0
    ldq = _rows(Q, Q.dtype, (total, Hq, D), "Q")
    ldo = _rows(out, Q.dtype, (total, Hq, D), "out")
    ldt = _rows(table, torch.int32, (B, width), "table")
    _dense(q_off, torch.int32, (B + 1,), "q_off")
    _dense(lens, torch.int32, (B,), "lens")
    f = _ftype(Q, "Q", short=True)
    pages, page = _kv4_cache(Kc, Vc, Kp, Vp, Hkv, D, Q)
    dev = _same_device(Q, Kc, Vc, Kp, Vp, table, q_off, lens, out)
    if lse is not None:
        _dense(lse, torch.float32, (total, Hq), "lse")
        _same_device(lse, out)
    max_q = total if max_q is None else max_q
    max_len = width * page if max_len is None else max_len
    lib = load()
    need = 0
    if workspace is None and Hkv > 0:
        need = lib.lb_attn_kv4_workspace(B, total, max_q, Hq, Hkv, D, max_len, window, 0)
    ws, size, kept = _scratch(workspace, need, Q, stream, "lb_attn_kv4")
    _raise(lib.lb_attn_kv4(Q.data_ptr(), ldq, Kc.data_ptr(), Vc.data_ptr(), Kp.data_ptr(), Vp.data_ptr(),
                           table.data_ptr(), ldt, width, q_off.data_ptr(), lens.data_ptr(), out.data_ptr(), ldo,
                           None if lse is None else lse.data_ptr(), B, total, max_q, Hq, Hkv, D, pages, page,
                           max_len, D ** -0.5 if scale is None else scale, window, int(causal), f, ws, size,
                           _raw_stream(stream, dev)), "lb_attn_kv4")
