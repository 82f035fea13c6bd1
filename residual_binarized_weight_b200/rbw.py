"""Thin ctypes binding of the C ABI in ``include/rbw.h`` (librbw.so).

Argument marshalling only: every step of the computation runs in the CUDA
library.  Tensors must be CUDA tensors on the current device; the calls are
issued on torch's current stream.  A missing library raises immediately
(there is no fallback path).
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librbw.so")

RB_OK, RB_ERR_ARG, RB_ERR_SHAPE, RB_ERR_ALIGN, RB_ERR_WORKSPACE, RB_ERR_UNSUPPORTED, RB_ERR_CUDA = range(7)
RB_DEV_NONFINITE, RB_DEV_RANGE, RB_DEV_TIMEOUT = 0x1, 0x2, 0x4
RB_F32, RB_BF16 = 0, 1
RB_LAUNCH_PDL = 0x1
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}

# name -> (restype, argtypes); the full exported surface of include/rbw.h
_vp, _i32, _sz, _u32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint
_i64 = ctypes.c_int64
SIGNATURES = {
    "rb_version": (_i32, []),
    "rb_status_string": (ctypes.c_char_p, [_i32]),
    "rb_packed_words": (_sz, [_i32, _i32, _i32]),
    "rb_pack": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp]),
    "rb_gemv_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "rb_gemv": (_i32, [_vp, _vp, _i32, _vp, _i32, _vp, _sz, _vp, _u32, _vp]),
    "rb_gemv_batch": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _u32, _vp]),
    "rb_gemm_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "rb_gemm": (_i32, [_vp, _vp, _i32, _vp, _i32, _vp, _sz, _vp, _u32, _vp]),
    "rb_gemm_wait_limit": (_i32, [_vp, _vp, _i32, _vp, _i32, _vp, _sz, _vp, _u32, ctypes.c_uint64, _vp]),
    "rb_gemm_noalloc": (_i32, [_vp, _vp, _i32, _vp, _i32, _vp, _u32, _vp]),
    "rb_transpose_planes": (_i32, [_vp, _vp, _vp]),
    "rb_rowmajor_words": (_sz, [_i32, _i32, _i32]),
    "rb_shard_rows": (_i32, [_vp, _i32, _i32, _vp, _vp, _vp]),
    "rb_planes_from_rowmajor": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp]),
    "rb_planes_to_rowmajor": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp]),
    "rb_qat_forward_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "rb_qat_forward": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _sz, _vp, _u32, _vp]),
    "rb_qat_backward_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "rb_qat_backward": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "rb_btc_index_bits": (_i32, [_i32]),
    "rb_btc_row_words": (_sz, [_i32, _i32]),
    "rb_btc_encode_workspace_bytes": (_sz, [_i32]),
    "rb_btc_encode": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "rb_btc_gemv_workspace_bytes": (_sz, [_i32, _i32]),
    "rb_btc_gemv": (_i32, [_vp, _vp, _vp, _i32, _vp, _sz, _vp, _u32, _vp]),
    "rb_btc_gemv_batch_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "rb_btc_gemv_batch": (_i32, [_vp, _vp, _vp, _i32, _i32, _vp, _sz, _vp, _u32, _vp]),
    "rb_svid_workspace_bytes": (_sz, [_i32, _i32]),
    "rb_svid_greedy": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "rb_svid_iterative_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "rb_svid_iterative": (_i32, [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp]),
    "rb_svid_pack_workspace_bytes": (_sz, [_i32, _i32, _i32]),
    "rb_svid_pack": (_i32, [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "rb_linear_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "rb_linear": (_i32, [_vp, _vp, _i64, _i32, _vp, _vp, _i64, _i32, _vp, _sz, _vp, _u32, _vp]),
    "rb_qat_linear_workspace_bytes": (_sz, [_i32, _i32, _i32, _i32]),
    "rb_qat_linear": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _i64, _i32, _vp, _vp, _i64, _i32, _vp, _sz, _vp,
                             _u32, _vp]),
    "rb_epilogue_backward_workspace_bytes": (_sz, [_i32, _i32]),
    "rb_epilogue_backward": (_i32, [_vp, _i32, _i32, _vp, _sz, _u32, _vp]),
    "rb_adamw_step": (_i32, [_vp, _i32, _vp, _vp, _u32, _vp]),
}


class RbLayer(ctypes.Structure):
    _fields_ = [("n_out", ctypes.c_int32), ("k_in", ctypes.c_int32), ("k_planes", ctypes.c_int32),
                ("reserved", ctypes.c_int32), ("planes", _vp), ("g16", _vp), ("h16", _vp)]


class RbBtcLayer(ctypes.Structure):
    _fields_ = [("n_out", ctypes.c_int32), ("k_in", ctypes.c_int32), ("k_planes", ctypes.c_int32),
                ("c_max", ctypes.c_int32), ("index_bits", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("codebooks", _vp), ("indices", _vp), ("g16", _vp), ("h16", _vp)]


class RbEpilogue(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("residual_dtype", ctypes.c_int32), ("bias", _vp), ("mul", _vp),
                ("residual", _vp), ("preact", _vp), ("ld_mul", _i64), ("ld_residual", _i64), ("ld_preact", _i64),
                ("reserved", _i64)]


class RbEpilogueGrad(ctypes.Structure):
    _fields_ = [("act", ctypes.c_int32), ("reserved", ctypes.c_int32), ("dY", _vp), ("preact", _vp), ("mul", _vp),
                ("dP", _vp), ("dmul", _vp), ("dbias", _vp), ("ld_dy", _i64), ("ld_preact", _i64), ("ld_mul", _i64),
                ("ld_dp", _i64), ("ld_dmul", _i64)]


class RbAdamWTensor(ctypes.Structure):
    _fields_ = [("n", _i64), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32),
                ("state_bits", ctypes.c_int32), ("reserved", ctypes.c_int32), ("lr", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("param", _vp), ("grad", _vp), ("exp_avg", _vp),
                ("exp_avg_sq", _vp), ("exp_avg_scale", _vp), ("exp_avg_sq_scale", _vp)]


class RbAdamW(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double), ("step", _i64),
                ("seed", ctypes.c_uint32), ("reserved", ctypes.c_uint32), ("step_dev", _vp), ("lr_scale", _vp),
                ("grad_scale", _vp)]


_lib = None


def lib():
    """Load librbw.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("librbw.so not found at %s: run residual_binarized_weight_b200/build.py" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


class RbError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__("%s failed: %s" % (fn, lib().rb_status_string(status).decode()))


def _check(fn, status):
    if status != RB_OK:
        raise RbError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _on(stream):
    """Where a call on `stream` allocates: in that stream's memory if one is given, so that what the call makes for itself
    is not given out again before the call has run."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _empty(shape, dtype, device, stream=None):
    """A result of a call on `stream`, kept until the current stream, which may read it, is done with it as well."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with _on(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if t.is_cuda:
        t.record_stream(torch.cuda.current_stream(t.device))
    return t


def packed_words(n_out, k_in, k_planes):
    return int(lib().rb_packed_words(n_out, k_in, k_planes))


class PackedLayer:
    """Device tensors of one packed layer (owns them) plus its rb_layer_t view."""

    def __init__(self, n_out, k_in, k_planes, device="cuda", g16=None, h16=None, planes=None, stream=None):
        """New planes and scale tensors (for use on `stream`) unless existing ones are passed to share."""
        nw = packed_words(n_out, k_in, k_planes)
        if nw == 0:
            raise ValueError("invalid layer shape")
        self.n_out, self.k_in, self.k_planes = n_out, k_in, k_planes
        self.planes = _empty(nw, torch.int32, device, stream) if planes is None else planes
        if self.planes.numel() != nw or self.planes.element_size() != 4 or not self.planes.is_contiguous():
            raise ValueError("planes do not match the layer shape")
        self.g16 = _empty((k_planes, n_out), torch.float16, device, stream) if g16 is None else g16
        self.h16 = _empty((k_planes, k_in), torch.float16, device, stream) if h16 is None else h16
        if tuple(self.g16.shape) != (k_planes, n_out) or tuple(self.h16.shape) != (k_planes, k_in):
            raise ValueError("scale tensors do not match the layer shape")
        if any(t.dtype not in (torch.float16, torch.int16, torch.uint16) or not t.is_contiguous() for t in (self.g16, self.h16)):
            raise ValueError("scale tensors: expected contiguous torch.float16, or its bits in 16-bit integers")

    def struct(self):
        return RbLayer(self.n_out, self.k_in, self.k_planes, 0, self.planes.data_ptr(),
                       self.g16.data_ptr(), self.h16.data_ptr())

    def packed_bytes(self):
        return self.planes.numel() * 4


def pack(W, g, h, k_planes, out: PackedLayer | None = None, dev_status=None, stream=None):
    """rb_pack: W fp32 [N][K], g fp32 [k][N], h fp32 [k][K] (CUDA) -> PackedLayer."""
    N, K = W.shape
    out = out or PackedLayer(N, K, k_planes, W.device, stream=stream)
    st = lib().rb_pack(_ptr(W), _ptr(g), _ptr(h), N, K, k_planes, _ptr(out.planes), _ptr(out.g16),
                       _ptr(out.h16), _ptr(dev_status), _stream(stream))
    _check("rb_pack", st)
    return out


def gemv_workspace_bytes(n_out, k_in, k_planes, M):
    return int(lib().rb_gemv_workspace_bytes(n_out, k_in, k_planes, M))


def gemm_workspace_bytes(n_out, k_in, k_planes, M):
    return int(lib().rb_gemm_workspace_bytes(n_out, k_in, k_planes, M))


def svid_workspace_bytes(n_out, k_in):
    return int(lib().rb_svid_workspace_bytes(n_out, k_in))


def workspace(nbytes, device="cuda", stream=None):
    """Zero-filled device workspace (uint8) of at least nbytes (16-byte aligned), for a call on `stream`."""
    with _on(stream):
        return torch.zeros(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def _apply(fn_name, layer: PackedLayer, X, Y, ws, flags, dev_status, stream):
    M = X.shape[0]
    ydt = RB_BF16 if Y.dtype == torch.bfloat16 else RB_F32
    L = layer.struct()
    wsp, wsb = (None, 0) if ws is None else (_ptr(ws), ws.numel() * ws.element_size())
    st = getattr(lib(), fn_name)(ctypes.byref(L), _ptr(X), M, _ptr(Y), ydt, wsp, wsb,
                                 _ptr(dev_status), flags, _stream(stream))
    _check(fn_name, st)
    return Y


def gemv(layer: PackedLayer, X, Y=None, ws=None, flags=0, dev_status=None, stream=None, y_dtype=torch.float32):
    """rb_gemv: X bf16 [M][K] (M <= 64) -> Y [M][N] (fp32 or bf16)."""
    if Y is None:
        Y = _empty((X.shape[0], layer.n_out), y_dtype, X.device, stream)
    return _apply("rb_gemv", layer, X, Y, ws, flags, dev_status, stream)


def gemv_batch(layers, Xs, Ys, flags=0, dev_status=None, stream=None):
    """rb_gemv_batch: independent layers of one shape; Xs[j] bf16 [M][K], Ys[j] [M][N] (CUDA tensors)."""
    n = len(layers)
    structs = (RbLayer * n)(*[L.struct() for L in layers])
    lp = (ctypes.POINTER(RbLayer) * n)(*[ctypes.pointer(structs[j]) for j in range(n)])
    xp = (ctypes.c_void_p * n)(*[X.data_ptr() for X in Xs])
    yp = (ctypes.c_void_p * n)(*[Y.data_ptr() for Y in Ys])
    M = Xs[0].shape[0]
    ydt = RB_BF16 if Ys[0].dtype == torch.bfloat16 else RB_F32
    st = lib().rb_gemv_batch(ctypes.cast(lp, ctypes.c_void_p), ctypes.cast(xp, ctypes.c_void_p),
                             ctypes.cast(yp, ctypes.c_void_p), n, M, ydt, _ptr(dev_status), flags, _stream(stream))
    _check("rb_gemv_batch", st)
    return Ys


def gemm(layer: PackedLayer, X, Y=None, ws=None, flags=0, dev_status=None, stream=None, y_dtype=torch.float32):
    """rb_gemm: X bf16 [M][K] -> Y [M][N] (fp32 or bf16) on the tcgen05 tensor cores."""
    if Y is None:
        Y = _empty((X.shape[0], layer.n_out), y_dtype, X.device, stream)
    return _apply("rb_gemm", layer, X, Y, ws, flags, dev_status, stream)


def gemm_wait_limit(layer: PackedLayer, X, wait_limit_ns, Y=None, ws=None, flags=0, dev_status=None, stream=None,
                    y_dtype=torch.float32):
    """rb_gemm_wait_limit: rb_gemm with a caller-chosen bound (ns) on every device-side wait."""
    if Y is None:
        Y = _empty((X.shape[0], layer.n_out), y_dtype, X.device, stream)
    L = layer.struct()
    ydt = RB_BF16 if Y.dtype == torch.bfloat16 else RB_F32
    wsp, wsb = (None, 0) if ws is None else (_ptr(ws), ws.numel() * ws.element_size())
    st = lib().rb_gemm_wait_limit(ctypes.byref(L), _ptr(X), X.shape[0], _ptr(Y), ydt, wsp, wsb, _ptr(dev_status),
                                  flags, int(wait_limit_ns), _stream(stream))
    _check("rb_gemm_wait_limit", st)
    return Y


def gemm_noalloc(layer: PackedLayer, X, Y=None, flags=0, dev_status=None, stream=None, y_dtype=torch.float32):
    """rb_gemm_noalloc: rb_gemm without a workspace (fixed 32 MiB library scratch; see include/rbw.h)."""
    if Y is None:
        Y = _empty((X.shape[0], layer.n_out), y_dtype, X.device, stream)
    L = layer.struct()
    ydt = RB_BF16 if Y.dtype == torch.bfloat16 else RB_F32
    st = lib().rb_gemm_noalloc(ctypes.byref(L), _ptr(X), X.shape[0], _ptr(Y), ydt, _ptr(dev_status), flags,
                               _stream(stream))
    _check("rb_gemm_noalloc", st)
    return Y


def transpose(layer: PackedLayer, out: PackedLayer | None = None, stream=None):
    """rb_transpose_planes: the K x N layer of What^T (new planes, or out's; the
    scale tensors are shared with `layer`, exchanged).  Its forward product is
    the input gradient: gemv/gemm(transpose(layer), dY) = dY . What."""
    if out is None:
        out = PackedLayer(layer.k_in, layer.n_out, layer.k_planes, layer.planes.device, g16=layer.h16, h16=layer.g16,
                          stream=stream)
    elif (out.n_out, out.k_in, out.k_planes) != (layer.k_in, layer.n_out, layer.k_planes):
        raise ValueError("out is not shaped as the transposed layer")
    else:
        out.g16, out.h16 = layer.h16, layer.g16
    L = layer.struct()
    st = lib().rb_transpose_planes(ctypes.byref(L), _ptr(out.planes), _stream(stream))
    _check("rb_transpose_planes", st)
    return out


def rowmajor_words(n_out, k_in, k_planes):
    return int(lib().rb_rowmajor_words(n_out, k_in, k_planes))


def planes_from_rowmajor(rowmajor, n_out, k_in, k_planes, out: PackedLayer | None = None, stream=None):
    """rb_planes_from_rowmajor: plain [k][N][K/32] LSB-first words (int32 CUDA tensor)
    -> a PackedLayer whose planes hold them in the storage layout (scales left to the caller)."""
    out = out or PackedLayer(n_out, k_in, k_planes, rowmajor.device, stream=stream)
    st = lib().rb_planes_from_rowmajor(_ptr(rowmajor), n_out, k_in, k_planes, _ptr(out.planes), _stream(stream))
    _check("rb_planes_from_rowmajor", st)
    return out


def planes_to_rowmajor(layer: PackedLayer, out=None, stream=None):
    """rb_planes_to_rowmajor: the layer's planes as plain [k][N][K/32] LSB-first words (int32)."""
    n = rowmajor_words(layer.n_out, layer.k_in, layer.k_planes)
    out = out if out is not None else _empty(n, torch.int32, layer.planes.device, stream)
    st = lib().rb_planes_to_rowmajor(_ptr(layer.planes), layer.n_out, layer.k_in, layer.k_planes, _ptr(out),
                                     _stream(stream))
    _check("rb_planes_to_rowmajor", st)
    return out


def qat_forward_workspace_bytes(n_out, k_in, k_planes, M):
    return int(lib().rb_qat_forward_workspace_bytes(n_out, k_in, k_planes, M))


def qat_forward(W, g, h, k_planes, X, Y=None, ws=None, flags=0, dev_status=None, stream=None,
                y_dtype=torch.float32):
    """rb_qat_forward: Y = X What^T, planes derived from fp32 W into the workspace, fp32 scales (CUDA tensors)."""
    N, K = W.shape
    M = X.shape[0]
    if Y is None:
        Y = _empty((M, N), y_dtype, W.device, stream)
    ws = ws if ws is not None else workspace(qat_forward_workspace_bytes(N, K, k_planes, M), W.device, stream)
    ydt = RB_BF16 if Y.dtype == torch.bfloat16 else RB_F32
    st = lib().rb_qat_forward(_ptr(W), _ptr(g), _ptr(h), N, K, k_planes, _ptr(X), M, _ptr(Y), ydt, _ptr(ws),
                              ws.numel(), _ptr(dev_status), flags, _stream(stream))
    _check("rb_qat_forward", st)
    return Y


def qat_backward(layer: PackedLayer, g, h, X, dY, dW=None, dg=None, dh=None, ws=None, dev_status=None,
                 stream=None):
    """rb_qat_backward: (dW [N][K], dg [k][N], dh [k][K]) fp32 from the layer's planes, fp32 scales
    g [k][N], h [k][K], X bf16 [M][K] and dY bf16 [M][N] (CUDA tensors)."""
    N, K, k = layer.n_out, layer.k_in, layer.k_planes
    dev = layer.planes.device
    dW = dW if dW is not None else _empty((N, K), torch.float32, dev, stream)
    dg = dg if dg is not None else _empty((k, N), torch.float32, dev, stream)
    dh = dh if dh is not None else _empty((k, K), torch.float32, dev, stream)
    nb = int(lib().rb_qat_backward_workspace_bytes(N, K, k))
    ws = ws if ws is not None else workspace(nb, dev, stream)
    st = lib().rb_qat_backward(_ptr(layer.planes), _ptr(g), _ptr(h), N, K, k, _ptr(X), _ptr(dY), X.shape[0],
                               _ptr(dW), _ptr(dg), _ptr(dh), _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream))
    _check("rb_qat_backward", st)
    return dW, dg, dh


def svid_greedy(W, k_planes, iters=20, ws=None, stream=None):
    """rb_svid_greedy: fp32 W [N][K] (CUDA) -> (g [k][N], h [k][K]) fp32."""
    N, K = W.shape
    g = _empty((k_planes, N), torch.float32, W.device, stream)
    h = _empty((k_planes, K), torch.float32, W.device, stream)
    ws = ws if ws is not None else workspace(svid_workspace_bytes(N, K), W.device, stream)
    st = lib().rb_svid_greedy(_ptr(W), N, K, k_planes, iters, _ptr(g), _ptr(h), _ptr(ws),
                              ws.numel(), _stream(stream))
    _check("rb_svid_greedy", st)
    return g, h


def svid_iterative(W, k_planes, sweeps=20, iters=20, ws=None, stream=None):
    """rb_svid_iterative: greedy scales refined by Gauss-Seidel sweeps; fp32 W [N][K] (CUDA)."""
    N, K = W.shape
    g = _empty((k_planes, N), torch.float32, W.device, stream)
    h = _empty((k_planes, K), torch.float32, W.device, stream)
    nbytes = int(lib().rb_svid_iterative_workspace_bytes(N, K, k_planes))
    ws = ws if ws is not None else workspace(nbytes, W.device, stream)
    st = lib().rb_svid_iterative(_ptr(W), N, K, k_planes, sweeps, iters, _ptr(g), _ptr(h), _ptr(ws),
                                 ws.numel(), _stream(stream))
    _check("rb_svid_iterative", st)
    return g, h


def svid_pack(W, k_planes, sweeps=0, iters=20, out: PackedLayer | None = None, ws=None, dev_status=None,
              stream=None):
    """rb_svid_pack: fp32 W [N][K] (CUDA) -> (PackedLayer, g, h): SVID scales (greedy when sweeps = 0,
    else iterative) and the packed planes, in one device-side call."""
    N, K = W.shape
    out = out or PackedLayer(N, K, k_planes, W.device, stream=stream)
    g = _empty((k_planes, N), torch.float32, W.device, stream)
    h = _empty((k_planes, K), torch.float32, W.device, stream)
    nbytes = int(lib().rb_svid_pack_workspace_bytes(N, K, k_planes))
    ws = ws if ws is not None else workspace(nbytes, W.device, stream)
    st = lib().rb_svid_pack(_ptr(W), N, K, k_planes, sweeps, iters, _ptr(g), _ptr(h), _ptr(out.planes),
                            _ptr(out.g16), _ptr(out.h16), _ptr(ws), ws.numel(), _ptr(dev_status), _stream(stream))
    _check("rb_svid_pack", st)
    return out, g, h


def shard_bounds(n_out, world, rank):
    """Rows [row0, row1) of rank `rank` in a row-parallel split of n_out rows over
    `world` ranks: contiguous ranges starting on 32-row tiles, as even as that allows."""
    tiles = (n_out + 31) // 32
    t0, t1 = tiles * rank // world, tiles * (rank + 1) // world
    return min(32 * t0, n_out), min(32 * t1, n_out)


def shard_rows(layer: PackedLayer, row0, rows, stream=None):
    """rb_shard_rows: rows [row0, row0 + rows) of `layer` as a PackedLayer sharing its h16."""
    out = PackedLayer(rows, layer.k_in, layer.k_planes, layer.planes.device, h16=layer.h16, stream=stream)
    L = layer.struct()
    st = lib().rb_shard_rows(ctypes.byref(L), row0, rows, _ptr(out.planes), _ptr(out.g16), _stream(stream))
    _check("rb_shard_rows", st)
    return out


# ---------------------------------------------------------------- binary codebook
class BtcLayer:
    """Device tensors of a binary-codebook layer (owns the codebooks and index streams; shares g16, h16)."""

    def __init__(self, n_out, k_in, k_planes, c_max, g16, h16, device="cuda", stream=None):
        self.n_out, self.k_in, self.k_planes, self.c_max = n_out, k_in, k_planes, c_max
        self.index_bits = int(lib().rb_btc_index_bits(c_max))
        self.row_words = int(lib().rb_btc_row_words(k_in, self.index_bits))
        if self.index_bits == 0 or self.row_words == 0:
            raise ValueError("invalid codebook layer shape")
        with _on(stream):
            self.codebooks = torch.zeros(k_planes, c_max, dtype=torch.int16, device=device)
            self.indices = torch.zeros(k_planes, n_out, self.row_words, dtype=torch.int32, device=device)
            self.sizes = torch.zeros(k_planes, 4, dtype=torch.int32, device=device)   # c of each plane in column 0
        self.g16, self.h16 = g16, h16

    def struct(self):
        return RbBtcLayer(self.n_out, self.k_in, self.k_planes, self.c_max, self.index_bits, 0,
                          self.codebooks.data_ptr(), self.indices.data_ptr(), self.g16.data_ptr(),
                          self.h16.data_ptr())

    def index_bytes(self):
        return self.indices.numel() * 4


def btc_encode(layer: PackedLayer, c_max, iters=10, stream=None):
    """rb_btc_encode for every plane of a packed layer -> BtcLayer."""
    out = BtcLayer(layer.n_out, layer.k_in, layer.k_planes, c_max, layer.g16, layer.h16, layer.planes.device, stream)
    ws = workspace(int(lib().rb_btc_encode_workspace_bytes(c_max)), layer.planes.device, stream)
    L = layer.struct()
    for i in range(layer.k_planes):
        st = lib().rb_btc_encode(ctypes.byref(L), i, c_max, iters, _ptr(out.codebooks[i]), _ptr(out.sizes[i]),
                                 _ptr(out.indices[i]), _ptr(ws), ws.numel(), _stream(stream))
        _check("rb_btc_encode", st)
    return out


def btc_gemv(layer: BtcLayer, X, Y=None, ws=None, flags=0, stream=None, y_dtype=torch.float32):
    """rb_btc_gemv: X bf16 [1][K] (or [K]) -> Y [1][N]."""
    if Y is None:
        Y = _empty((1, layer.n_out), y_dtype, X.device, stream)
    ws = ws if ws is not None else workspace(int(lib().rb_btc_gemv_workspace_bytes(layer.n_out, layer.k_in)),
                                             X.device, stream)
    L = layer.struct()
    ydt = RB_BF16 if Y.dtype == torch.bfloat16 else RB_F32
    st = lib().rb_btc_gemv(ctypes.byref(L), _ptr(X), _ptr(Y), ydt, _ptr(ws), ws.numel(), None, flags,
                           _stream(stream))
    _check("rb_btc_gemv", st)
    return Y


def btc_gemv_batch(layers, Xs, Ys, ws=None, flags=0, stream=None):
    """rb_btc_gemv_batch: codebook layers of one shape; Xs[j] bf16 [1][K], Ys[j] [1][N] (CUDA tensors)."""
    n = len(layers)
    structs = (RbBtcLayer * n)(*[L.struct() for L in layers])
    lp = (ctypes.POINTER(RbBtcLayer) * n)(*[ctypes.pointer(structs[j]) for j in range(n)])
    xp = (ctypes.c_void_p * n)(*[X.data_ptr() for X in Xs])
    yp = (ctypes.c_void_p * n)(*[Y.data_ptr() for Y in Ys])
    L0 = layers[0]
    ws = ws if ws is not None else workspace(
        int(lib().rb_btc_gemv_batch_workspace_bytes(L0.n_out, L0.k_in, n)), Xs[0].device, stream)
    ydt = RB_BF16 if Ys[0].dtype == torch.bfloat16 else RB_F32
    st = lib().rb_btc_gemv_batch(lp, xp, yp, n, ydt, _ptr(ws), ws.numel(), None, flags, _stream(stream))
    _check("rb_btc_gemv_batch", st)
    return Ys


# ---------------------------------------------------------------- epilogue gradient
def _scratch(nbytes, device, stream):
    """A call's own workspace, not cleared."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    with _on(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


_BF16 = (torch.bfloat16,)


def _matrix(t, name, M, N, dev, dtypes=_BF16):
    """(address, row stride) of an [M][N] tensor with unit column stride on device `dev`, or (None, 0)."""
    if t is None:
        return None, 0
    if t.dtype not in dtypes or t.shape != (M, N):
        raise ValueError("%s: expected a [%d, %d] tensor of %s" % (name, M, N, " or ".join(map(str, dtypes))))
    if t.get_device() != dev:
        raise ValueError("%s: expected a tensor on the current CUDA device" % name)
    ld, step = t.stride()
    if M == 1:                                             # the stride of a lone row says nothing
        ld = N
    if (step != 1 and N > 1) or ld < N:
        raise ValueError("%s: columns must be contiguous and rows must not overlap" % name)
    return t.data_ptr(), ld


def _vector(t, name, n, dev, dtype=torch.float32, shape=None):
    """Address of a contiguous tensor of n elements, or of the given shape."""
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError("%s: expected a tensor of shape %s" % (name, shape))
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous():
        raise ValueError("%s: expected a contiguous %s tensor of %d elements" % (name, dtype, n))
    if t.get_device() != dev:
        raise ValueError("%s: expected a tensor on the current CUDA device" % name)
    return t.data_ptr()


def _status(t, dev):
    """Address of a device status word, or None."""
    if t is None:
        return None
    if t.dtype != torch.int32 or t.numel() < 1 or t.get_device() != dev:
        raise ValueError("dev_status: expected an int32 tensor on the current CUDA device")
    return t.data_ptr()


def _workspace(t, dev):
    """(address, bytes) of a workspace."""
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError("ws: expected a contiguous tensor on the current CUDA device")
    return t.data_ptr(), t.nbytes


def _current(stream):
    """(current device, address of the given stream or of torch's current one), without making Stream objects."""
    dev = torch.cuda.current_device()
    return dev, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


_Y_TYPES = (torch.float32, torch.bfloat16)


def _epilogue(M, N, dev, bias, act, mul, residual, preact):
    b = None if bias is None else _vector(bias, "bias", N, dev)
    mp, ldm = (None, 0) if mul is None else _matrix(mul, "mul", M, N, dev)
    rp, ldr = (None, 0) if residual is None else _matrix(residual, "residual", M, N, dev, _Y_TYPES)
    pp, ldp = (None, 0) if preact is None else _matrix(preact, "preact", M, N, dev)
    rdt = RB_BF16 if residual is not None and residual.dtype is torch.bfloat16 else RB_F32
    return RbEpilogue(ACTS[act], rdt, b, mp, rp, pp, ldm, ldr, ldp, 0)


def linear_workspace_bytes(n_out, k_in, k_planes, M):
    return int(lib().rb_linear_workspace_bytes(n_out, k_in, k_planes, M))


def linear(layer: PackedLayer, X, Y=None, bias=None, act="none", mul=None, residual=None, preact=None, ws=None,
           flags=0, dev_status=None, stream=None, y_dtype=torch.bfloat16):
    """rb_linear: Y = act(X What^T + bias) * mul + residual for X bf16 [M][K], any M.  bias fp32 [N]; mul bf16,
    residual bf16 or fp32, preact (out: the pre-activation) bf16, all [M][N], rows may be strided; residual may be Y."""
    M, N, K = X.shape[0], layer.n_out, layer.k_in
    dev, st = _current(stream)
    if Y is None:
        Y = _empty((M, N), y_dtype, X.device, stream)
    xp, ldx = _matrix(X, "X", M, K, dev)
    yp, ldy = _matrix(Y, "Y", M, N, dev, _Y_TYPES)
    E = _epilogue(M, N, dev, bias, act, mul, residual, preact)
    if ws is None:
        ws = _scratch(linear_workspace_bytes(N, K, layer.k_planes, M), X.device, stream)
    if not layer.planes.get_device() == layer.g16.get_device() == layer.h16.get_device() == dev:
        raise ValueError("layer: expected tensors on the current CUDA device")
    wsp, wsb = _workspace(ws, dev)
    st = lib().rb_linear(ctypes.byref(layer.struct()), xp, ldx, M, ctypes.byref(E), yp, ldy,
                         RB_BF16 if Y.dtype is torch.bfloat16 else RB_F32, wsp, wsb,
                         _status(dev_status, dev), flags, st)
    if st != RB_OK:
        raise RbError("rb_linear", st)
    return Y


def qat_linear_workspace_bytes(n_out, k_in, k_planes, M):
    return int(lib().rb_qat_linear_workspace_bytes(n_out, k_in, k_planes, M))


def qat_linear(W, g, h, k_planes, X, Y=None, bias=None, act="none", mul=None, residual=None, preact=None, ws=None,
               flags=0, dev_status=None, stream=None, y_dtype=torch.bfloat16):
    """rb_qat_linear: as linear, with the planes derived from fp32 W [N][K] and the fp32 scales g [k][N], h [k][K]."""
    N, K = W.shape
    M = X.shape[0]
    if Y is None:
        Y = _empty((M, N), y_dtype, X.device, stream)
    dev, st = _current(stream)
    xp, ldx = _matrix(X, "X", M, K, dev)
    yp, ldy = _matrix(Y, "Y", M, N, dev, _Y_TYPES)
    E = _epilogue(M, N, dev, bias, act, mul, residual, preact)
    if ws is None:
        ws = _scratch(qat_linear_workspace_bytes(N, K, k_planes, M), X.device, stream)
    wsp, wsb = _workspace(ws, dev)
    st = lib().rb_qat_linear(_vector(W, "W", N * K, dev), _vector(g, "g", k_planes * N, dev, shape=(k_planes, N)),
                             _vector(h, "h", k_planes * K, dev, shape=(k_planes, K)), N, K, k_planes, xp, ldx, M, ctypes.byref(E), yp, ldy,
                             RB_BF16 if Y.dtype is torch.bfloat16 else RB_F32, wsp, wsb,
                             _status(dev_status, dev), flags, st)
    _check("rb_qat_linear", st)
    return Y


def epilogue_backward_workspace_bytes(M, n_out):
    return int(lib().rb_epilogue_backward_workspace_bytes(M, n_out))


def epilogue_backward(dY, preact, act="none", mul=None, bias=True, dP=None, dmul=None, dbias=None, ws=None, flags=0,
                      stream=None):
    """rb_epilogue_backward: (dP, dmul, dbias) of Y = act(P) * mul + residual from dY and P, bf16 [M][N] (rows
    may be strided).  dmul is None without mul, dbias (fp32 [N]) without bias; the residual's gradient is dY."""
    M, N = dY.shape
    if dP is None:
        dP = _empty((M, N), torch.bfloat16, dY.device, stream)
    if dmul is None and mul is not None:
        dmul = _empty((M, N), torch.bfloat16, dY.device, stream)
    if dbias is None and bias:
        dbias = _empty(N, torch.float32, dY.device, stream)
    dev, st = _current(stream)
    wsp, wsb = None, 0
    if dbias is not None:
        if ws is None:
            ws = _scratch(epilogue_backward_workspace_bytes(M, N), dY.device, stream)
        wsp, wsb = _workspace(ws, dev)
    yp, ldy = _matrix(dY, "dY", M, N, dev)
    pp, ldp = _matrix(preact, "preact", M, N, dev)
    up, ldu = _matrix(mul, "mul", M, N, dev)
    dpp, lddp = _matrix(dP, "dP", M, N, dev)
    dup, lddu = _matrix(dmul, "dmul", M, N, dev)
    G = RbEpilogueGrad(ACTS[act], 0, yp, pp, up, dpp, dup, None if dbias is None else _vector(dbias, "dbias", N, dev),
                       ldy, ldp, ldu, lddp, lddu)
    st = lib().rb_epilogue_backward(ctypes.byref(G), M, N, wsp, wsb, flags, st)
    _check("rb_epilogue_backward", st)
    return dP, dmul, dbias


# ---------------------------------------------------------------- optimizer
ADAMW_BLOCK = 256                # elements that share a scale of the 8-bit states


class AdamWTensor:
    """One tensor of an AdamW step: a parameter, its gradient and its states (contiguous CUDA tensors).

    32-bit states: exp_avg and exp_avg_sq fp32.  8-bit: both torch.float8_e4m3fn (exp_avg_sq holding square
    roots) with fp32 scales of ceil(n / 256) elements.  `new_state` makes fresh ones.  Any of them, the rate and the
    decay may be assigned anew between steps."""

    _edits = 0                   # assignments to any AdamWTensor, so that a step sees at once that there were none

    def __init__(self, param, grad, exp_avg, exp_avg_sq, exp_avg_scale=None, exp_avg_sq_scale=None, lr=1e-3,
                 weight_decay=0.0):
        self.param, self.grad, self.exp_avg, self.exp_avg_sq = param, grad, exp_avg, exp_avg_sq
        self.exp_avg_scale, self.exp_avg_sq_scale = exp_avg_scale, exp_avg_sq_scale
        self.lr, self.weight_decay = lr, weight_decay
        self.check()

    def __setattr__(self, name, value):
        AdamWTensor._edits += 1
        d = self.__dict__
        d["edits"] = d.get("edits", 0) + 1
        if name not in ("grad", "lr", "weight_decay"):      # what a step may well replace each time
            d["made"] = d["edits"]
        d[name] = value

    @property
    def state_bits(self):
        return 32 if self.exp_avg is None or self.exp_avg.dtype == torch.float32 else 8

    @property
    def device(self):
        return self.param.get_device()

    def _fits(self, name, types, want):
        t, p = self.__dict__[name], self.param
        if t is None or t.dtype not in types or t.numel() != want or not t.is_contiguous():
            raise ValueError("%s: expected %d contiguous elements of %s" % (name, want, " or ".join(map(str, types))))
        if t.get_device() != p.get_device():
            raise ValueError("a parameter, its gradient and its states are on one device")
        if name[-5:] != "scale" and t.dim() > 1 and p.dim() > 1 and t.shape != p.shape:
            raise ValueError("%s: expected the parameter's shape, or one dimension" % name)

    def check_grad(self):
        self._fits("grad", _Y_TYPES, self.param.numel())

    def check(self):
        n, bits = self.param.numel(), self.state_bits
        self._fits("param", _Y_TYPES, n)
        self.check_grad()
        for name in ("exp_avg", "exp_avg_sq"):
            self._fits(name, (torch.float32 if bits == 32 else torch.float8_e4m3fn,), n)
        if bits == 8:
            for name in ("exp_avg_scale", "exp_avg_sq_scale"):
                self._fits(name, (torch.float32,), (n + ADAMW_BLOCK - 1) // ADAMW_BLOCK)

    @staticmethod
    def new_state(param, bits=32):
        """Keyword arguments exp_avg, exp_avg_sq (and scales) of a fresh state."""
        if bits not in (8, 32):
            raise ValueError("states have 8 or 32 bits")
        dt = torch.float32 if bits == 32 else torch.float8_e4m3fn
        s = {k: torch.zeros(param.numel(), dtype=torch.float32 if bits == 32 else torch.uint8,
                            device=param.device).view(dt) for k in ("exp_avg", "exp_avg_sq")}
        if bits == 8:
            blocks = (param.numel() + ADAMW_BLOCK - 1) // ADAMW_BLOCK
            s |= {k: torch.zeros(blocks, dtype=torch.float32, device=param.device)
                  for k in ("exp_avg_scale", "exp_avg_sq_scale")}
        return s

    def struct(self):
        p = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        dt = lambda t: RB_BF16 if t.dtype == torch.bfloat16 else RB_F32  # noqa: E731
        return RbAdamWTensor(self.param.numel(), dt(self.param), dt(self.grad), self.state_bits, 0, self.lr,
                             self.weight_decay, p(self.param), p(self.grad), p(self.exp_avg), p(self.exp_avg_sq),
                             p(self.exp_avg_scale), p(self.exp_avg_sq_scale))


class AdamW:
    """rb_adamw_step over a fixed list of AdamWTensor (one call for all of them).  The table of addresses, rates and
    decays that the library takes is kept from step to step and follows what is assigned to the AdamWTensors;
    `refresh` makes it anew, which is needed where a tensor's memory is swapped beneath it (`t.data = ..`, `set_`)."""

    def __init__(self, tensors, beta1=0.9, beta2=0.999, eps=1e-8, seed=0):
        self.tensors = tuple(tensors)
        self.hyper = RbAdamW(beta1, beta2, eps, 0, seed & 0xFFFFFFFF, 0, None, None, None)
        self.refresh()

    def refresh(self):
        self._table = (RbAdamWTensor * len(self.tensors))()
        self._taken = [(-1, -1)] * len(self.tensors)        # each tensor's counts of assignments when its row was made
        self._follow()

    def _follow(self):
        if not self.tensors or any(t.device != self.tensors[0].device for t in self.tensors):
            raise ValueError("expected tensors of one device, at least one")
        edits = AdamWTensor._edits
        for i, t in enumerate(self.tensors):
            now, taken = (t.made, t.edits), self._taken[i]
            if now == taken:
                continue
            if t.made == taken[0]:                          # the gradient, the rate or the decay
                t.check_grad()
                row = self._table[i]
                row.grad, row.grad_dtype = t.grad.data_ptr(), RB_BF16 if t.grad.dtype == torch.bfloat16 else RB_F32
                row.lr, row.weight_decay = t.lr, t.weight_decay
            else:
                t.check()
                self._table[i] = t.struct()
            self._taken[i] = now
        self._edits = edits

    def step(self, step, lr_scale=None, grad_scale=None, dev_status=None, flags=0, stream=None):
        """One step; `step` is its number (from 1), or an int32 CUDA tensor that holds it (for captured graphs).
        lr_scale and grad_scale: fp32 CUDA tensors of one element that multiply every lr and every gradient."""
        H = self.hyper
        if self._edits != AdamWTensor._edits:
            self._follow()
        dev, st = _current(stream)
        if self.tensors[0].device != dev:
            raise ValueError("the tensors are not on the current CUDA device")
        if isinstance(step, torch.Tensor):
            H.step, H.step_dev = 0, _vector(step, "step", 1, dev, torch.int32)
        else:
            H.step, H.step_dev = step, None
        H.lr_scale = None if lr_scale is None else _vector(lr_scale, "lr_scale", 1, dev)
        H.grad_scale = None if grad_scale is None else _vector(grad_scale, "grad_scale", 1, dev)
        st = lib().rb_adamw_step(self._table, len(self.tensors), ctypes.byref(H),
                                 _status(dev_status, dev), flags, st)
        _check("rb_adamw_step", st)
