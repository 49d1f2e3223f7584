"""Python binding of liblcvq.so, the LC-VQ hot path on MI355X (gfx950).

Argument marshalling only: every function here checks tensor dtypes, devices and
contiguity, then passes raw device pointers and the current HIP stream to the C ABI
declared in include/lcvq.h. All arithmetic runs in the library's HIP kernels; if the
library is missing the import of any entry point raises.

Names follow the C ABI (lcvq_quantize, lcvq_pack2b, lcvq_unpack2b, lcvq_linear_fwd,
lcvq_linear_bwd, lcvq_linear_bwd_dge, lcvq_gemv2b, lcvq_gemv2b_noalloc,
lcvq_gemv2b_batched, lcvq_hessian, lcvq_ptq_init, lcvq_mx_quantize, lcvq_mx_dequantize,
lcvq_mxfp4_gemm, lcvq_mxfp4_gemv, lcvq_linear_bwd_ckpt8, lcvq_silu_gate_fwd,
lcvq_silu_gate_bwd and the *_workspace_size helpers).
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblcvq.so")

LCVQ_F32, LCVQ_BF16 = 0, 1
LCVQ_MXFP4, LCVQ_MXINT8 = 0, 1
_STATUS = {0: "LCVQ_OK", 1: "LCVQ_ERR_NULL", 2: "LCVQ_ERR_SHAPE", 3: "LCVQ_ERR_D",
           4: "LCVQ_ERR_DTYPE", 5: "LCVQ_ERR_ALIGN", 6: "LCVQ_ERR_WORKSPACE", 7: "LCVQ_ERR_HIP",
           8: "LCVQ_ERR_VALUE", 9: "LCVQ_ERR_SCRATCH"}

_lib = None


class GemvMatrix(ctypes.Structure):
    """lcvq_gemv2b_matrix: one matrix of a batched decode product."""
    _fields_ = [("packed", ctypes.c_void_p), ("A16", ctypes.c_void_p), ("B16", ctypes.c_void_p),
                ("Y", ctypes.c_void_p), ("N", ctypes.c_int64), ("layout", ctypes.c_int32)]


class LcvqError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)} "
                         f"({lib().lcvq_status_string(status).decode()})")


def lib():
    """The loaded liblcvq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m bit_weight_only_lc_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        f32 = ctypes.c_float
        L.lcvq_status_string.restype = ctypes.c_char_p
        L.lcvq_status_string.argtypes = [i32]
        sigs = {
            "lcvq_quantize": [vp, i64, i64, vp, vp, vp, vp],
            "lcvq_pack2b": [vp, i64, i64, vp, vp],
            "lcvq_unpack2b": [vp, i64, i64, vp, vp],
            "lcvq_linear_fwd": [vp, i32, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp, vp,
                                sz, vp],
            "lcvq_linear_bwd": [vp, vp, i32, i64, i64, i64, i32, vp, vp, vp, vp, vp, vp, vp,
                                vp, vp, sz, vp],
            "lcvq_linear_bwd_dge": [vp, vp, i32, i64, i64, i64, i32, vp, vp, vp, f32, vp, vp,
                                    vp, vp, vp, vp, vp, sz, vp],
            "lcvq_gemv2b": [vp, i64, i64, i64, i32, vp, vp, vp, vp, vp, sz, vp],
            "lcvq_gemv2b_shuffled": [vp, i64, i64, i64, i32, vp, vp, vp, vp, vp, sz, vp],
            "lcvq_gemv2b_shuffle": [vp, i64, i64, vp, vp],
            "lcvq_gemv2b_noalloc": [vp, i64, i64, i64, i32, vp, vp, vp, vp, vp],
            "lcvq_hessian": [vp, i64, i64, vp, vp],
            "lcvq_mx_quantize": [vp, i32, i64, i64, i32, vp, vp, vp],
            "lcvq_mx_dequantize": [vp, vp, i64, i64, i32, vp, i32, vp],
            "lcvq_mxfp4_gemm": [vp, vp, i64, i64, i64, vp, vp, vp, i32, vp, sz, vp],
            "lcvq_mxfp4_gemv": [vp, i64, i64, i64, vp, vp, vp, vp],
            "lcvq_linear_bwd_ckpt8": [vp, vp, vp, i32, i64, i64, i64, i32, vp, vp, vp, vp, vp,
                                      vp, vp, vp, vp, sz, vp],
            "lcvq_silu_gate_fwd": [vp, vp, i32, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp],
            "lcvq_silu_gate_bwd": [vp, i32, i64, i64, vp, vp, vp, vp, vp, vp, vp],
            "lcvq_read_probe": [vp, i64, vp, vp],
            "lcvq_mfma_probe": [i64, vp, vp],
            "lcvq_ptq_init": [vp, vp, i64, i64, f32, i32, vp, vp, vp, vp, vp, vp, sz, vp],
        }
        for name, args in sigs.items():
            f = getattr(L, name)
            f.restype = i32
            f.argtypes = args
        for name in ("lcvq_linear_fwd_workspace_size", "lcvq_linear_bwd_workspace_size",
                     "lcvq_linear_bwd_ckpt8_workspace_size"):
            f = getattr(L, name)
            f.restype = sz
            f.argtypes = [i64, i64, i64, i32]
        L.lcvq_gemv2b_batched.restype = i32
        L.lcvq_gemv2b_batched.argtypes = [vp, i64, i64, i32, ctypes.POINTER(GemvMatrix), i32,
                                          vp, sz, vp]
        L.lcvq_mxfp4_gemm_workspace_size.restype = sz
        L.lcvq_mxfp4_gemm_workspace_size.argtypes = [i64, i64, i64]
        L.lcvq_ptq_workspace_size.restype = sz
        L.lcvq_ptq_workspace_size.argtypes = [i64, i64]
        L.lcvq_gemv2b_workspace_size.restype = sz
        L.lcvq_gemv2b_workspace_size.argtypes = [i64, i64, i64, i32]
        L.lcvq_profile_next.restype = i32
        L.lcvq_profile_next.argtypes = [i32, vp, vp]
        _lib = L
    return _lib


def _p(t):
    return None if t is None else t.data_ptr()


def _check(t, name, dtype=None, device=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _current_stream(i):
    return torch.cuda.current_stream(i).cuda_stream


# The handle alone of GPU i's current stream: building a torch.cuda.Stream object costs 2 us. A
# torch without GPU support lacks the first name; the module is imported there all the same.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _stream(dev):
    return _raw_stream(dev.index)


def _ok(status, where):
    if status != 0:
        raise LcvqError(status, where)


def _dt(t):
    if t.dtype == torch.bfloat16:
        return LCVQ_BF16
    if t.dtype == torch.float32:
        return LCVQ_F32
    raise TypeError(f"activations must be bfloat16 or float32, got {t.dtype}")


# ------------------------------------------------------------------ workspace sizes
def lcvq_linear_fwd_workspace_size(M, N, K, d):
    return int(lib().lcvq_linear_fwd_workspace_size(M, N, K, d))


def lcvq_linear_bwd_workspace_size(M, N, K, d):
    return int(lib().lcvq_linear_bwd_workspace_size(M, N, K, d))


def lcvq_gemv2b_workspace_size(M, N, K, d):
    return int(lib().lcvq_gemv2b_workspace_size(M, N, K, d))


def lcvq_linear_bwd_ckpt8_workspace_size(M, N, K, d):
    return int(lib().lcvq_linear_bwd_ckpt8_workspace_size(M, N, K, d))


def lcvq_mxfp4_gemm_workspace_size(M, N, K):
    return int(lib().lcvq_mxfp4_gemm_workspace_size(M, N, K))


# ------------------------------------------------------------------ entry points
def lcvq_quantize(Wp, z_u8=None, packed=None, mask=None):
    _check(Wp, "Wp", torch.float32)
    dev = Wp.device
    for t, n in ((z_u8, "z_u8"), (packed, "packed"), (mask, "mask")):
        _check(t, n, torch.uint8, dev)
    N, K = Wp.shape
    _ok(lib().lcvq_quantize(_p(Wp), N, K, _p(z_u8), _p(packed), _p(mask), _stream(dev)),
        "lcvq_quantize")


def lcvq_pack2b(z_u8, packed):
    _check(z_u8, "z_u8", torch.uint8)
    _check(packed, "packed", torch.uint8, z_u8.device)
    N, K = z_u8.shape
    _ok(lib().lcvq_pack2b(_p(z_u8), N, K, _p(packed), _stream(z_u8.device)), "lcvq_pack2b")


def lcvq_unpack2b(packed, z_u8):
    _check(packed, "packed", torch.uint8)
    _check(z_u8, "z_u8", torch.uint8, packed.device)
    N, K = z_u8.shape
    _ok(lib().lcvq_unpack2b(_p(packed), N, K, _p(z_u8), _stream(packed.device)),
        "lcvq_unpack2b")


def lcvq_linear_fwd(X, Wp, A, B, d, Y, packed_out, mask_out, What_out=None, workspace=None):
    _check(X, "X", (torch.bfloat16, torch.float32))
    dev = X.device
    _check(Wp, "Wp", torch.float32, dev)
    _check(A, "A", torch.float32, dev)
    _check(B, "B", torch.float32, dev)
    _check(Y, "Y", X.dtype, dev)
    _check(packed_out, "packed_out", torch.uint8, dev)
    _check(mask_out, "mask_out", torch.uint8, dev)
    _check(What_out, "What_out", torch.float32, dev)
    M, K = X.shape
    N = Wp.shape[0]
    if workspace is None:
        workspace = torch.empty(max(lcvq_linear_fwd_workspace_size(M, N, K, d), 1),
                                dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", torch.uint8, dev)
    _ok(lib().lcvq_linear_fwd(_p(X), _dt(X), M, N, K, d, _p(Wp), _p(A), _p(B), _p(Y),
                              _p(packed_out), _p(mask_out), _p(What_out), _p(workspace),
                              workspace.numel(), _stream(dev)), "lcvq_linear_fwd")


def lcvq_linear_bwd(dY, X, packed, mask, A, B, d, dX, dWp, dA, dB, workspace=None):
    _check(dY, "dY", (torch.bfloat16, torch.float32))
    dev = dY.device
    _check(X, "X", dY.dtype, dev)
    _check(packed, "packed", torch.uint8, dev)
    _check(mask, "mask", torch.uint8, dev)
    _check(A, "A", torch.float32, dev)
    _check(B, "B", torch.float32, dev)
    _check(dX, "dX", dY.dtype, dev)
    _check(dWp, "dWp", torch.float32, dev)
    _check(dA, "dA", torch.float32, dev)
    _check(dB, "dB", torch.float32, dev)
    M, N = dY.shape
    K = X.shape[1]
    if workspace is None:
        workspace = torch.empty(max(lcvq_linear_bwd_workspace_size(M, N, K, d), 1),
                                dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", torch.uint8, dev)
    _ok(lib().lcvq_linear_bwd(_p(dY), _p(X), _dt(dY), M, N, K, d, _p(packed), _p(mask),
                              _p(A), _p(B), _p(dX), _p(dWp), _p(dA), _p(dB), _p(workspace),
                              workspace.numel(), _stream(dev)), "lcvq_linear_bwd")


def lcvq_linear_bwd_dge(dY, X, packed, mask, Wp, alpha, A, B, d, dX, dWp, dA, dB,
                        workspace=None):
    _check(dY, "dY", (torch.bfloat16, torch.float32))
    dev = dY.device
    _check(X, "X", dY.dtype, dev)
    _check(packed, "packed", torch.uint8, dev)
    _check(mask, "mask", torch.uint8, dev)
    _check(Wp, "Wp", torch.float32, dev)
    _check(A, "A", torch.float32, dev)
    _check(B, "B", torch.float32, dev)
    _check(dX, "dX", dY.dtype, dev)
    _check(dWp, "dWp", torch.float32, dev)
    _check(dA, "dA", torch.float32, dev)
    _check(dB, "dB", torch.float32, dev)
    M, N = dY.shape
    K = X.shape[1]
    if workspace is None:
        workspace = torch.empty(max(lcvq_linear_bwd_workspace_size(M, N, K, d), 1),
                                dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", torch.uint8, dev)
    _ok(lib().lcvq_linear_bwd_dge(_p(dY), _p(X), _dt(dY), M, N, K, d, _p(packed), _p(mask),
                                  _p(Wp), float(alpha), _p(A), _p(B), _p(dX), _p(dWp), _p(dA),
                                  _p(dB), _p(workspace), workspace.numel(), _stream(dev)),
        "lcvq_linear_bwd_dge")


def lcvq_gemv2b(X, packed, A16, B16, d, Y, workspace=None):
    _gemv2b("lcvq_gemv2b", X, packed, A16, B16, d, Y, workspace)


def lcvq_gemv2b_noalloc(X, packed, A16, B16, d, Y):
    """lcvq_gemv2b on the library's fixed scratch: no workspace, nothing allocated."""
    _check(X, "X", torch.bfloat16)
    dev = X.device
    _check(packed, "packed", torch.uint8, dev)
    _check(A16, "A16", torch.float16, dev)
    _check(B16, "B16", torch.float16, dev)
    _check(Y, "Y", torch.bfloat16, dev)
    M, K = X.shape
    N = packed.shape[0]
    _ok(lib().lcvq_gemv2b_noalloc(_p(X), M, N, K, d, _p(packed), _p(A16), _p(B16), _p(Y),
                                  _stream(dev)), "lcvq_gemv2b_noalloc")


def lcvq_gemv2b_shuffled(X, codes, A16, B16, d, Y, workspace=None):
    """codes: the decode layout written by lcvq_gemv2b_shuffle, held as uint8 [N, K/4]."""
    _gemv2b("lcvq_gemv2b_shuffled", X, codes, A16, B16, d, Y, workspace)


def lcvq_gemv2b_shuffle(packed, codes):
    dev = packed.device
    _check(packed, "packed", torch.uint8, dev)
    _check(codes, "codes", torch.uint8, dev)
    if codes.shape != packed.shape:
        raise ValueError("codes must have the shape of packed")
    N, K4 = packed.shape
    _ok(lib().lcvq_gemv2b_shuffle(_p(packed), N, K4 * 4, _p(codes), _stream(dev)),
        "lcvq_gemv2b_shuffle")


def _gemv2b(name, X, packed, A16, B16, d, Y, workspace):
    _check(X, "X", torch.bfloat16)
    dev = X.device
    _check(packed, "packed", torch.uint8, dev)
    _check(A16, "A16", torch.float16, dev)
    _check(B16, "B16", torch.float16, dev)
    _check(Y, "Y", torch.bfloat16, dev)
    M, K = X.shape
    N = packed.shape[0]
    if workspace is None:
        workspace = torch.empty(max(lcvq_gemv2b_workspace_size(M, N, K, d), 1),
                                dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", torch.uint8, dev)
    _ok(getattr(lib(), name)(_p(X), M, N, K, d, _p(packed), _p(A16), _p(B16), _p(Y),
                             _p(workspace), workspace.numel(), _stream(dev)), name)


def lcvq_gemv2b_batched(X, mats, d, workspace=None):
    """mats: list of (packed, A16, B16, Y) or (packed, A16, B16, Y, layout) sharing the
    input X; layout 1 means codes in the decode layout of lcvq_gemv2b_shuffle."""
    _check(X, "X", torch.bfloat16)
    dev = X.device
    M, K = X.shape
    arr = (GemvMatrix * max(len(mats), 1))()
    nmax = 16
    for i, m in enumerate(mats):
        pk, a16, b16, y = m[:4]
        layout = m[4] if len(m) > 4 else 0
        _check(pk, "packed", torch.uint8, dev)
        _check(a16, "A16", torch.float16, dev)
        _check(b16, "B16", torch.float16, dev)
        _check(y, "Y", torch.bfloat16, dev)
        arr[i] = GemvMatrix(pk.data_ptr(), a16.data_ptr(), b16.data_ptr(), y.data_ptr(),
                            pk.shape[0], int(layout))
        nmax = max(nmax, pk.shape[0])
    if workspace is None:
        workspace = torch.empty(max(lcvq_gemv2b_workspace_size(M, nmax, K, d), 1),
                                dtype=torch.uint8, device=dev)
    _check(workspace, "workspace", torch.uint8, dev)
    _ok(lib().lcvq_gemv2b_batched(_p(X), M, K, d, arr, len(mats), _p(workspace),
                                  workspace.numel(), _stream(dev)), "lcvq_gemv2b_batched")


# ------------------------------------------------------------------ block-scaled formats
_ACT = (torch.bfloat16, torch.float32)
_BF16, _F32, _U8, _I8 = torch.bfloat16, torch.float32, torch.uint8, torch.int8


def _need(t, name, dtype, i, *shape):
    """A contiguous tensor of this type and shape on GPU i. Where all is well this is one
    test; a decode step makes dozens of these calls, and each is as long as a small kernel."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                and t.get_device() == i):
            return
    except AttributeError:
        pass
    if t is None:
        raise ValueError(f"{name} is missing")
    _check(t, name, dtype, torch.device("cuda", i))
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")


def _need_mx(codes, scales, name, fmt, M, K, i):
    """Codes and scales of a block-scaled [M, K] matrix."""
    if fmt == LCVQ_MXFP4:
        _need(codes, name, _U8, i, M, K // 2)
    elif fmt == LCVQ_MXINT8:
        _need(codes, name, _I8, i, M, K)
    else:
        raise ValueError(f"unknown block format {fmt}")
    _need(scales, name + "_scales", _U8, i, M, K // 32)


def _mat(t, name, dtypes=_ACT):
    """A two-dimensional contiguous GPU tensor: its GPU and shape."""
    try:
        i = t.get_device()
        if t.dtype in dtypes and i >= 0 and t.is_contiguous():
            rows, cols = t.shape
            return i, rows, cols
    except (AttributeError, ValueError):
        pass
    if t is None:
        raise ValueError(f"{name} is missing")
    _check(t, name, dtypes)
    raise ValueError(f"{name} has {t.dim()} dimensions, expected 2")


def _need_workspace(t, i):
    if t.dtype is _U8 and t.get_device() == i and t.is_contiguous():
        return
    _check(t, "workspace", _U8, torch.device("cuda", i))


def lcvq_mx_quantize(X, fmt, codes, scales):
    """X [M, K] (bf16 or float32) -> codes and scales of fmt (LCVQ_MXFP4 or LCVQ_MXINT8)."""
    i, M, K = _mat(X, "X")
    _need_mx(codes, scales, "X", fmt, M, K, i)
    _ok(lib().lcvq_mx_quantize(X.data_ptr(), _dt(X), M, K, fmt, codes.data_ptr(),
                               scales.data_ptr(), _raw_stream(i)), "lcvq_mx_quantize")


def lcvq_mx_dequantize(codes, scales, fmt, out):
    """The values that codes and scales stand for, into out [M, K] (bf16 or float32)."""
    i, M, K = _mat(out, "out")
    _need_mx(codes, scales, "X", fmt, M, K, i)
    _ok(lib().lcvq_mx_dequantize(codes.data_ptr(), scales.data_ptr(), M, K, fmt, out.data_ptr(),
                                 _dt(out), _raw_stream(i)), "lcvq_mx_dequantize")


def lcvq_mxfp4_gemm(Xc, Xs, Wc, Ws, Y, workspace=None):
    """Y [M, N] (bf16 or float32) = X W^T, X [M, K] and W [N, K] in MXFP4. (No workspace is
    used; one that is given is checked.)"""
    i, M, N = _mat(Y, "Y")
    K = _mat(Wc, "W", (_U8,))[2] * 2
    _need_mx(Xc, Xs, "X", LCVQ_MXFP4, M, K, i)
    _need_mx(Wc, Ws, "W", LCVQ_MXFP4, N, K, i)
    if workspace is not None:
        _need_workspace(workspace, i)
    _ok(lib().lcvq_mxfp4_gemm(Xc.data_ptr(), Xs.data_ptr(), M, N, K, Wc.data_ptr(),
                              Ws.data_ptr(), Y.data_ptr(), _dt(Y), _p(workspace),
                              0 if workspace is None else workspace.numel(), _raw_stream(i)),
        "lcvq_mxfp4_gemm")


def lcvq_mxfp4_gemv(X, Wc, Ws, Y):
    """Y [M, N] = X W^T for 1..16 rows of bf16 X [M, K] and W [N, K] in MXFP4."""
    i, M, K = _mat(X, "X", (_BF16,))
    N = _mat(Wc, "W", (_U8,))[1]
    _need_mx(Wc, Ws, "W", LCVQ_MXFP4, N, K, i)
    _need(Y, "Y", _BF16, i, M, N)
    _ok(lib().lcvq_mxfp4_gemv(X.data_ptr(), M, N, K, Wc.data_ptr(), Ws.data_ptr(), Y.data_ptr(),
                              _raw_stream(i)), "lcvq_mxfp4_gemv")


def lcvq_linear_bwd_ckpt8(dY, Xc, Xs, packed, mask, A, B, d, dX, dWp, dA, dB, workspace=None):
    """lcvq_linear_bwd with X as an LCVQ_MXINT8 checkpoint (codes Xc, scales Xs)."""
    i, M, N = _mat(dY, "dY")
    K = _mat(packed, "packed", (_U8,))[2] * 4
    _need_mx(Xc, Xs, "X", LCVQ_MXINT8, M, K, i)
    _need(packed, "packed", _U8, i, N, K // 4)
    _need(mask, "mask", _U8, i, N, K // 8)
    _need(A, "A", _F32, i, d, d)
    _need(B, "B", _F32, i, d)
    if dX is not None:
        _need(dX, "dX", dY.dtype, i, M, K)
    _need(dWp, "dWp", _F32, i, N, K)
    _need(dA, "dA", _F32, i, d, d)
    _need(dB, "dB", _F32, i, d)
    if workspace is None:
        workspace = torch.empty(max(lcvq_linear_bwd_ckpt8_workspace_size(M, N, K, d), 1),
                                dtype=torch.uint8, device=dY.device)
    _need_workspace(workspace, i)
    _ok(lib().lcvq_linear_bwd_ckpt8(dY.data_ptr(), Xc.data_ptr(), Xs.data_ptr(), _dt(dY), M, N,
                                    K, d, packed.data_ptr(), mask.data_ptr(), A.data_ptr(),
                                    B.data_ptr(), _p(dX), dWp.data_ptr(), dA.data_ptr(),
                                    dB.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                    _raw_stream(i)), "lcvq_linear_bwd_ckpt8")


def lcvq_silu_gate_fwd(G, U, H, Gc=None, Gs=None, Uc=None, Us=None, Hc=None, Hs=None):
    """H = silu(G) * U, and LCVQ_MXINT8 checkpoints of G, U and H where buffers are given."""
    i, M, F = _mat(G, "G")
    _need(U, "U", G.dtype, i, M, F)
    _need(H, "H", G.dtype, i, M, F)
    for c, s, n in ((Gc, Gs, "G"), (Uc, Us, "U"), (Hc, Hs, "H")):
        if c is not None or s is not None:
            _need_mx(c, s, n, LCVQ_MXINT8, M, F, i)
    _ok(lib().lcvq_silu_gate_fwd(G.data_ptr(), U.data_ptr(), _dt(G), M, F, H.data_ptr(), _p(Gc),
                                 _p(Gs), _p(Uc), _p(Us), _p(Hc), _p(Hs), _raw_stream(i)),
        "lcvq_silu_gate_fwd")


def lcvq_silu_gate_bwd(dH, Gc, Gs, Uc, Us, dG, dU):
    """dG, dU of the gate from dH and the checkpoints of G and U."""
    i, M, F = _mat(dH, "dH")
    _need_mx(Gc, Gs, "G", LCVQ_MXINT8, M, F, i)
    _need_mx(Uc, Us, "U", LCVQ_MXINT8, M, F, i)
    _need(dG, "dG", dH.dtype, i, M, F)
    _need(dU, "dU", dH.dtype, i, M, F)
    _ok(lib().lcvq_silu_gate_bwd(dH.data_ptr(), _dt(dH), M, F, Gc.data_ptr(), Gs.data_ptr(),
                                 Uc.data_ptr(), Us.data_ptr(), dG.data_ptr(), dU.data_ptr(),
                                 _raw_stream(i)), "lcvq_silu_gate_bwd")


def lcvq_mfma_probe(iters, sink):
    """Measurement helper: iters * 2^29 flops of bf16 MFMA issue into sink (int32 [1024])."""
    _check(sink, "sink", torch.int32)
    _ok(lib().lcvq_mfma_probe(int(iters), _p(sink), _stream(sink.device)), "lcvq_mfma_probe")


def lcvq_read_probe(buf, sink):
    """Measurement helper: stream buf once (uint8 device tensor) into sink (int32 [1024])."""
    _check(buf, "buf", torch.uint8)
    _check(sink, "sink", torch.int32, buf.device)
    _ok(lib().lcvq_read_probe(_p(buf), buf.numel(), _p(sink), _stream(buf.device)),
        "lcvq_read_probe")


def lcvq_hessian(X, H):
    """H = X^T X (X bf16 [M, K], H float32 [K, K])."""
    _check(X, "X", torch.bfloat16)
    _check(H, "H", torch.float32, X.device)
    M, K = X.shape
    _ok(lib().lcvq_hessian(_p(X), M, K, _p(H), _stream(X.device)), "lcvq_hessian")


def lcvq_ptq_workspace_size(N, K):
    return int(lib().lcvq_ptq_workspace_size(N, K))


def lcvq_ptq_init(H, W0, damp, iters, packed_out, sb_out, obj_out=None, U_out=None,
                  D_out=None, workspace=None):
    _check(H, "H", torch.float32)
    dev = H.device
    _check(W0, "W0", torch.float32, dev)
    _check(packed_out, "packed_out", torch.uint8, dev)
    _check(sb_out, "sb_out", torch.float32, dev)
    for t, n in ((obj_out, "obj_out"), (U_out, "U_out"), (D_out, "D_out")):
        _check(t, n, torch.float32, dev)
    N, K = W0.shape
    if workspace is None:
        workspace = torch.empty(max(lcvq_ptq_workspace_size(N, K), 1), dtype=torch.uint8,
                                device=dev)
    _check(workspace, "workspace", torch.uint8, dev)
    _ok(lib().lcvq_ptq_init(_p(H), _p(W0), N, K, float(damp), int(iters), _p(packed_out),
                            _p(sb_out), _p(obj_out), _p(U_out), _p(D_out), _p(workspace),
                            workspace.numel(), _stream(dev)), "lcvq_ptq_init")


def ptq_init(X, W0, damp=0.01, iters=4, want_ud=False):
    """Allocating helper: H = X^T X, then the initialisation. Returns a dict with H, the
    packed codes, s, b, the objective history (and U, D with want_ud)."""
    dev = X.device
    M, K = X.shape
    N = W0.shape[0]
    H = torch.empty((K, K), dtype=torch.float32, device=dev)
    lcvq_hessian(X, H)
    out = {"H": H,
           "packed": torch.empty((N, K // 4), dtype=torch.uint8, device=dev),
           "sb": torch.empty(2, dtype=torch.float32, device=dev),
           "obj": torch.empty(2 * iters, dtype=torch.float32, device=dev),
           "U": torch.empty((K, K), dtype=torch.float32, device=dev) if want_ud else None,
           "D": torch.empty(K, dtype=torch.float32, device=dev) if want_ud else None}
    lcvq_ptq_init(H, W0, damp, iters, out["packed"], out["sb"], out["obj"], out["U"], out["D"])
    return out


# ------------------------------------------------------------------ allocating helpers
def linear_fwd(X, Wp, A, B, d, want_what=False):
    """Allocates the outputs of lcvq_linear_fwd and returns them in a dict."""
    M, K = X.shape
    N = Wp.shape[0]
    dev = X.device
    out = {
        "Y": torch.empty((M, N), dtype=X.dtype, device=dev),
        "packed": torch.empty((N, K // 4), dtype=torch.uint8, device=dev),
        "mask": torch.empty((N, K // 8), dtype=torch.uint8, device=dev),
        "What": torch.empty((N, K), dtype=torch.float32, device=dev) if want_what else None,
    }
    lcvq_linear_fwd(X, Wp, A, B, d, out["Y"], out["packed"], out["mask"], out["What"])
    return out


def linear_bwd(dY, X, packed, mask, A, B, d, want_dx=True, dge_wp=None, dge_alpha=None):
    """Allocates the outputs of lcvq_linear_bwd (or, with dge_wp and dge_alpha, of
    lcvq_linear_bwd_dge) and returns them in a dict."""
    M, N = dY.shape
    K = X.shape[1]
    dev = dY.device
    out = {
        "dX": torch.empty((M, K), dtype=dY.dtype, device=dev) if want_dx else None,
        "dWp": torch.empty((N, K), dtype=torch.float32, device=dev),
        "dA": torch.empty((d, d), dtype=torch.float32, device=dev),
        "dB": torch.empty((d,), dtype=torch.float32, device=dev),
    }
    if dge_alpha is None:
        lcvq_linear_bwd(dY, X, packed, mask, A, B, d, out["dX"], out["dWp"], out["dA"],
                        out["dB"])
    else:
        lcvq_linear_bwd_dge(dY, X, packed, mask, dge_wp, dge_alpha, A, B, d, out["dX"],
                            out["dWp"], out["dA"], out["dB"])
    return out


def gemv2b(X, packed, A16, B16, d, shuffled=False):
    """Allocates Y; `shuffled` says that `packed` holds the decode layout."""
    M = X.shape[0]
    N = packed.shape[0]
    Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    (lcvq_gemv2b_shuffled if shuffled else lcvq_gemv2b)(X, packed, A16, B16, d, Y)
    return Y


def gemv2b_shuffle(packed):
    """Allocates and returns the decode layout of canonical packed codes."""
    codes = torch.empty_like(packed)
    lcvq_gemv2b_shuffle(packed, codes)
    return codes


def mx_empty(M, K, fmt, device):
    """Allocates the codes and scales of a block-scaled [M, K] matrix."""
    codes = torch.empty((M, K // 2) if fmt == LCVQ_MXFP4 else (M, K), device=device,
                        dtype=torch.uint8 if fmt == LCVQ_MXFP4 else torch.int8)
    return codes, torch.empty((M, K // 32), dtype=torch.uint8, device=device)


def mx_quantize(X, fmt):
    """Allocates and returns the codes and scales of X in fmt."""
    codes, scales = mx_empty(*X.shape, fmt, X.device)
    lcvq_mx_quantize(X, fmt, codes, scales)
    return codes, scales


def mx_dequantize(codes, scales, fmt, dtype=torch.bfloat16):
    """Allocates and returns the values that codes and scales stand for."""
    out = torch.empty((scales.shape[0], scales.shape[1] * 32), dtype=dtype, device=scales.device)
    lcvq_mx_dequantize(codes, scales, fmt, out)
    return out


def mxfp4_linear(X, Wc, Ws, quantize_x=None):
    """Y = X W^T (bf16) for a weight in MXFP4. X is 4 bits only where the caller says so:
    quantize_x True   X in MXFP4 too (bf16 or float32, lcvq_mxfp4_gemm)
    quantize_x False  X as it is, bf16, in one decode product (lcvq_mxfp4_gemv: 16 rows at most)
    quantize_x None   X as it is, bf16, any number of rows: one decode product, which reads
                      the weight once, for every 16."""
    M, N = X.shape[0], Wc.shape[0]
    Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    if quantize_x:
        lcvq_mxfp4_gemm(*mx_quantize(X, LCVQ_MXFP4), Wc, Ws, Y)
    elif quantize_x is None and M > 16:
        for m in range(0, M, 16):
            lcvq_mxfp4_gemv(X[m:m + 16], Wc, Ws, Y[m:m + 16])
    else:
        lcvq_mxfp4_gemv(X, Wc, Ws, Y)
    return Y


def linear_bwd_ckpt8(dY, Xc, Xs, packed, mask, A, B, d, want_dx=True):
    """Allocates the outputs of lcvq_linear_bwd_ckpt8 and returns them in a dict."""
    M, N = dY.shape
    K = Xc.shape[1]
    dev = dY.device
    out = {
        "dX": torch.empty((M, K), dtype=dY.dtype, device=dev) if want_dx else None,
        "dWp": torch.empty((N, K), dtype=torch.float32, device=dev),
        "dA": torch.empty((d, d), dtype=torch.float32, device=dev),
        "dB": torch.empty((d,), dtype=torch.float32, device=dev),
    }
    lcvq_linear_bwd_ckpt8(dY, Xc, Xs, packed, mask, A, B, d, out["dX"], out["dWp"], out["dA"],
                          out["dB"])
    return out


def silu_gate_fwd(G, U):
    """H = silu(G) * U with its three checkpoints, in a dict: H, and (codes, scales) pairs
    under "G8", "U8" and "H8"."""
    M, F = G.shape
    out = {"H": torch.empty_like(G)}
    for n in ("G8", "U8", "H8"):
        out[n] = mx_empty(M, F, LCVQ_MXINT8, G.device)
    lcvq_silu_gate_fwd(G, U, out["H"], *out["G8"], *out["U8"], *out["H8"])
    return out


def silu_gate_bwd(dH, G8, U8):
    """Allocates and returns dG, dU; G8, U8 are (codes, scales) pairs of the forward."""
    dG, dU = torch.empty_like(dH), torch.empty_like(dH)
    lcvq_silu_gate_bwd(dH, *G8, *U8, dG, dU)
    return dG, dU
