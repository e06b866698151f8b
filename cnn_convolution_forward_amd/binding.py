"""Thin ctypes binding to libconvfwd.so (argument marshalling only).

The functions named like the C ABI (``conv2d_fwd_bf16`` ...) take raw device
pointers (ints) and sizes, exactly as declared in ``include/conv_fwd.h``, and
return the status code.  The ``conv2d`` / ``conv3d`` / ``im2col`` helpers take
torch tensors that already live on the GPU, allocate the output with torch
(device memory and streams are all torch is used for), pass pointers and the
current HIP stream, and raise :class:`ConvError` on a non-OK status.  Every
arithmetic step runs in the library's HIP kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libconvfwd.so")

CONV_OK = 0
STATUS_NAMES = {0: "CONV_OK", 1: "CONV_ERR_NULL", 2: "CONV_ERR_PARAM", 3: "CONV_ERR_SHAPE",
                4: "CONV_ERR_OVERFLOW", 5: "CONV_ERR_ALIAS", 6: "CONV_ERR_WORKSPACE",
                7: "CONV_ERR_ALGO", 8: "CONV_ERR_HIP", 9: "CONV_ERR_SCRATCH"}
ALGO = {"auto": 0, "mfma": 1, "valu": 2, "winograd": 3}

# Every symbol include/conv_fwd.h declares.
EXPORTS = ("conv_out_dim", "conv_status_str", "conv_version",
           "conv2d_fwd_bf16", "conv2d_fwd_f32", "conv3d_fwd_bf16", "conv3d_fwd_f32",
           "conv2d_fwd_workspace_bytes", "conv2d_fwd_bf16_ws",
           "conv2d_pack_weights_bf16", "conv2d_fwd_bf16_prepacked", "conv2d_fwd_bf16_noalloc",
           "conv_im2col_bytes", "conv2d_im2col_bf16", "conv3d_im2col_bf16",
           "conv2d_fwd_bf16_explicit", "conv3d_fwd_bf16_explicit",
           "conv_out_dim_dilated", "conv_fwd_bf16", "conv_fwd_f32", "conv_xcol_bytes",
           "conv_im2col_bf16", "conv_fwd_explicit_bf16",
           "conv_bwd_data_workspace_bytes", "conv_bwd_data_bf16",
           "conv_bwd_weight_workspace_bytes", "conv_bwd_weight_bf16",
           "conv_fwd_ex_workspace_bytes", "conv_fwd_ex_bf16", "conv_fwd_ex_f32",
           "conv_causal_fwd", "conv_causal_bwd_workspace_bytes", "conv_causal_bwd", "conv_causal_step",
           "conv_scan_fwd_workspace_bytes", "conv_scan_fwd", "conv_scan_bwd_workspace_bytes", "conv_scan_bwd",
           "conv_scan_step", "conv_adamw_step", "conv_adamw_state_values")

LAYOUT = {"nchw": 0, "nhwc": 1}
OUT_DTYPE = {"f32": 0, "bf16": 1}


class ConvParams(ctypes.Structure):
    """conv_params_t: a general problem (dilation and groups)."""
    _fields_ = [(n, ctypes.c_int) for n in ("ndim", "N", "C_in", "D", "H", "W", "C_out", "K", "stride",
                                             "pad", "dilation", "groups")]


class ConvOptions(ctypes.Structure):
    """conv_options_t: layout of x and y, output dtype, ReLU."""
    _fields_ = [("layout", ctypes.c_int), ("out_dtype", ctypes.c_int), ("relu", ctypes.c_int)]


class SeqParams(ctypes.Structure):
    """conv_seq_t: a batch of sequences of tokens, equal or packed."""
    _fields_ = [("dtype", ctypes.c_int), ("B", ctypes.c_int), ("T", ctypes.c_int), ("C", ctypes.c_int),
                ("offsets", ctypes.c_void_p), ("tokens", ctypes.c_int64)]


class AdamwTensor(ctypes.Structure):
    """conv_adamw_tensor_t: one tensor's parameters, gradient and moments."""
    _fields_ = [("n", ctypes.c_int64)] + [(n, ctypes.c_void_p) for n in ("p", "g", "m", "v", "m_scale", "v_scale",
                                                                         "copy")] + [("weight_decay", ctypes.c_float)]


class AdamwOptions(ctypes.Structure):
    """conv_adamw_t: the step's rates and formats."""
    _fields_ = [(n, ctypes.c_double) for n in ("lr", "beta1", "beta2", "eps")] + \
        [("step", ctypes.c_int64), ("bits", ctypes.c_int), ("grad_dtype", ctypes.c_int), ("seed", ctypes.c_uint32),
         ("grad_scale", ctypes.c_void_p)]


class ConvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, STATUS_NAMES.get(status, status), status_str(status)))


_lib = None
_vp, _i, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t


def lib():
    """Load libconvfwd.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libconvfwd.so is not built (%s); run "
                              "`python -m cnn_convolution_forward_amd.build`" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        L.conv_out_dim.restype = _i64
        L.conv_out_dim.argtypes = [_i64] * 4
        L.conv_status_str.restype = ctypes.c_char_p
        L.conv_status_str.argtypes = [_i]
        L.conv_version.restype = _i
        L.conv_version.argtypes = []
        d2 = [_vp, _vp, _vp, _vp] + [_i] * 9 + [_vp]
        d3 = [_vp, _vp, _vp, _vp] + [_i] * 10 + [_vp]
        for name, args in (("conv2d_fwd_bf16", d2), ("conv2d_fwd_f32", d2),
                           ("conv3d_fwd_bf16", d3), ("conv3d_fwd_f32", d3)):
            getattr(L, name).restype = _i
            getattr(L, name).argtypes = args
        L.conv2d_fwd_workspace_bytes.restype = _sz
        L.conv2d_fwd_workspace_bytes.argtypes = [_i] * 9
        L.conv2d_fwd_bf16_ws.restype = _i
        L.conv2d_fwd_bf16_ws.argtypes = [_vp] * 5 + [_sz] + [_i] * 9 + [_vp]
        L.conv2d_pack_weights_bf16.restype = _i
        L.conv2d_pack_weights_bf16.argtypes = [_vp, _vp, _sz] + [_i] * 9 + [_vp]
        L.conv2d_fwd_bf16_prepacked.restype = _i
        L.conv2d_fwd_bf16_prepacked.argtypes = [_vp, _vp, _sz, _vp, _vp] + [_i] * 9 + [_vp]
        L.conv2d_fwd_bf16_noalloc.restype = _i
        L.conv2d_fwd_bf16_noalloc.argtypes = d2
        L.conv_im2col_bytes.restype = _sz
        L.conv_im2col_bytes.argtypes = [_i] * 9
        L.conv2d_im2col_bf16.restype = _i
        L.conv2d_im2col_bf16.argtypes = [_vp, _vp] + [_i] * 7 + [_vp]
        L.conv3d_im2col_bf16.restype = _i
        L.conv3d_im2col_bf16.argtypes = [_vp, _vp] + [_i] * 8 + [_vp]
        L.conv2d_fwd_bf16_explicit.restype = _i
        L.conv2d_fwd_bf16_explicit.argtypes = [_vp] * 5 + [_sz] + [_i] * 8 + [_vp]
        L.conv3d_fwd_bf16_explicit.restype = _i
        L.conv3d_fwd_bf16_explicit.argtypes = [_vp] * 5 + [_sz] + [_i] * 9 + [_vp]
        _pp = ctypes.POINTER(ConvParams)
        L.conv_out_dim_dilated.restype = _i64
        L.conv_out_dim_dilated.argtypes = [_i64] * 5
        for name in ("conv_fwd_bf16", "conv_fwd_f32"):
            getattr(L, name).restype = _i
            getattr(L, name).argtypes = [_pp, _vp, _vp, _vp, _vp, _i, _vp]
        L.conv_xcol_bytes.restype = _sz
        L.conv_xcol_bytes.argtypes = [_pp]
        L.conv_im2col_bf16.restype = _i
        L.conv_im2col_bf16.argtypes = [_pp, _vp, _vp, _vp]
        L.conv_fwd_explicit_bf16.restype = _i
        L.conv_fwd_explicit_bf16.argtypes = [_pp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        for name in ("conv_bwd_data_workspace_bytes", "conv_bwd_weight_workspace_bytes"):
            getattr(L, name).restype = _sz
            getattr(L, name).argtypes = [_pp]
        L.conv_bwd_data_bf16.restype = _i
        L.conv_bwd_data_bf16.argtypes = [_pp, _vp, _vp, _vp, _vp, _sz, _vp]
        L.conv_bwd_weight_bf16.restype = _i
        L.conv_bwd_weight_bf16.argtypes = [_pp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        _po = ctypes.POINTER(ConvOptions)
        L.conv_fwd_ex_workspace_bytes.restype = _sz
        L.conv_fwd_ex_workspace_bytes.argtypes = [_pp, _po, _i]
        L.conv_fwd_ex_bf16.restype = _i
        L.conv_fwd_ex_bf16.argtypes = [_pp, _po, _vp, _vp, _vp, _vp, _vp, _sz, _i, _vp]
        L.conv_fwd_ex_f32.restype = _i
        L.conv_fwd_ex_f32.argtypes = [_pp, _po, _vp, _vp, _vp, _vp, _i, _vp]
        _ps = ctypes.POINTER(SeqParams)
        _f = ctypes.c_float
        row = [_vp, _i64]                       # a tensor of rows and its row stride
        L.conv_causal_fwd.restype = _i
        L.conv_causal_fwd.argtypes = [_ps, _i, _i] + row + [_vp] * 3 + row + [_vp, _vp]
        L.conv_causal_bwd_workspace_bytes.restype = _sz
        L.conv_causal_bwd_workspace_bytes.argtypes = [_ps, _i]
        L.conv_causal_bwd.restype = _i
        L.conv_causal_bwd.argtypes = [_ps, _i, _i] + row + [_vp] * 3 + row * 2 + [_vp] * 4 + [_sz, _vp]
        L.conv_causal_step.restype = _i
        L.conv_causal_step.argtypes = [_ps, _i, _i] + row + [_vp] * 3 + row + [_vp]
        for name in ("conv_scan_fwd_workspace_bytes", "conv_scan_bwd_workspace_bytes"):
            getattr(L, name).restype = _sz
            getattr(L, name).argtypes = [_ps]
        L.conv_scan_fwd.restype = _i
        L.conv_scan_fwd.argtypes = [_ps, _f] + row * 3 + [_vp] * 2 + row + [_vp] * 3 + [_sz, _vp]
        L.conv_scan_bwd.restype = _i
        L.conv_scan_bwd.argtypes = [_ps, _f] + row * 3 + [_vp] * 2 + row + [_vp] + row * 3 + [_vp] * 3 + [_sz, _vp]
        L.conv_scan_step.restype = _i
        L.conv_scan_step.argtypes = [_ps, _f] + row * 3 + [_vp] * 2 + row + [_vp]
        L.conv_adamw_step.restype = _i
        L.conv_adamw_step.argtypes = [ctypes.POINTER(AdamwOptions), _vp, _i, _vp]
        L.conv_adamw_state_values.restype = _i
        L.conv_adamw_state_values.argtypes = [_vp, _i, _vp, _vp, _vp]
        _lib = L
    return _lib


# ---- the C ABI, same names, raw pointers -------------------------------------

def conv_out_dim(n, k, stride, pad):
    return int(lib().conv_out_dim(n, k, stride, pad))


def status_str(status):
    return lib().conv_status_str(int(status)).decode()


def conv_status_str(status):
    return status_str(status)


def conv_version():
    return int(lib().conv_version())


def conv2d_fwd_bf16(x, w, bias, y, N, C_in, H, W, C_out, K, stride, pad, algo=0, stream=None):
    return lib().conv2d_fwd_bf16(x, w, bias, y, N, C_in, H, W, C_out, K, stride, pad, algo, stream)


def conv2d_fwd_f32(x, w, bias, y, N, C_in, H, W, C_out, K, stride, pad, algo=0, stream=None):
    return lib().conv2d_fwd_f32(x, w, bias, y, N, C_in, H, W, C_out, K, stride, pad, algo, stream)


def conv3d_fwd_bf16(x, w, bias, y, N, C_in, D, H, W, C_out, K, stride, pad, algo=0, stream=None):
    return lib().conv3d_fwd_bf16(x, w, bias, y, N, C_in, D, H, W, C_out, K, stride, pad, algo, stream)


def conv3d_fwd_f32(x, w, bias, y, N, C_in, D, H, W, C_out, K, stride, pad, algo=0, stream=None):
    return lib().conv3d_fwd_f32(x, w, bias, y, N, C_in, D, H, W, C_out, K, stride, pad, algo, stream)


def conv2d_fwd_workspace_bytes(N, C_in, H, W, C_out, K, stride, pad, algo=0):
    return int(lib().conv2d_fwd_workspace_bytes(N, C_in, H, W, C_out, K, stride, pad, algo))


def conv2d_pack_weights_bf16(w, ws, ws_bytes, N, C_in, H, W, C_out, K, stride, pad, algo=0, stream=None):
    return lib().conv2d_pack_weights_bf16(w, ws, ws_bytes, N, C_in, H, W, C_out, K, stride, pad, algo, stream)


def conv2d_fwd_bf16_prepacked(x, ws, ws_bytes, bias, y, N, C_in, H, W, C_out, K, stride, pad, algo=0,
                              stream=None):
    return lib().conv2d_fwd_bf16_prepacked(x, ws, ws_bytes, bias, y, N, C_in, H, W, C_out, K, stride, pad,
                                           algo, stream)


def conv2d_fwd_bf16_ws(x, w, bias, y, ws, ws_bytes, N, C_in, H, W, C_out, K, stride, pad, algo=0,
                       stream=None):
    return lib().conv2d_fwd_bf16_ws(x, w, bias, y, ws, ws_bytes, N, C_in, H, W, C_out, K, stride, pad,
                                    algo, stream)


def conv2d_fwd_bf16_noalloc(x, w, bias, y, N, C_in, H, W, C_out, K, stride, pad, algo=0, stream=None):
    return lib().conv2d_fwd_bf16_noalloc(x, w, bias, y, N, C_in, H, W, C_out, K, stride, pad, algo, stream)


def conv_im2col_bytes(ndim, N, C_in, D, H, W, K, stride, pad):
    return int(lib().conv_im2col_bytes(ndim, N, C_in, D, H, W, K, stride, pad))


def conv2d_im2col_bf16(x, xcol, N, C_in, H, W, K, stride, pad, stream=None):
    return lib().conv2d_im2col_bf16(x, xcol, N, C_in, H, W, K, stride, pad, stream)


def conv3d_im2col_bf16(x, xcol, N, C_in, D, H, W, K, stride, pad, stream=None):
    return lib().conv3d_im2col_bf16(x, xcol, N, C_in, D, H, W, K, stride, pad, stream)


def conv2d_fwd_bf16_explicit(x, w, bias, y, ws, ws_bytes, N, C_in, H, W, C_out, K, stride, pad,
                             stream=None):
    return lib().conv2d_fwd_bf16_explicit(x, w, bias, y, ws, ws_bytes, N, C_in, H, W, C_out, K,
                                          stride, pad, stream)


def conv3d_fwd_bf16_explicit(x, w, bias, y, ws, ws_bytes, N, C_in, D, H, W, C_out, K, stride, pad,
                             stream=None):
    return lib().conv3d_fwd_bf16_explicit(x, w, bias, y, ws, ws_bytes, N, C_in, D, H, W, C_out, K,
                                          stride, pad, stream)


def _pref(params):
    return None if params is None else ctypes.byref(params)


def conv_out_dim_dilated(n, k, stride, pad, dilation):
    return int(lib().conv_out_dim_dilated(n, k, stride, pad, dilation))


def conv_fwd_bf16(params, x, w, bias, y, algo=0, stream=None):
    return lib().conv_fwd_bf16(_pref(params), x, w, bias, y, algo, stream)


def conv_fwd_f32(params, x, w, bias, y, algo=0, stream=None):
    return lib().conv_fwd_f32(_pref(params), x, w, bias, y, algo, stream)


def conv_xcol_bytes(params):
    return int(lib().conv_xcol_bytes(_pref(params)))


def conv_im2col_bf16(params, x, xcol, stream=None):
    return lib().conv_im2col_bf16(_pref(params), x, xcol, stream)


def conv_fwd_explicit_bf16(params, x, w, bias, y, ws, ws_bytes, stream=None):
    return lib().conv_fwd_explicit_bf16(_pref(params), x, w, bias, y, ws, ws_bytes, stream)


def conv_bwd_data_workspace_bytes(params):
    return int(lib().conv_bwd_data_workspace_bytes(_pref(params)))


def conv_bwd_data_bf16(params, dout, w, dx, ws, ws_bytes, stream=None):
    return lib().conv_bwd_data_bf16(_pref(params), dout, w, dx, ws, ws_bytes, stream)


def conv_bwd_weight_workspace_bytes(params):
    return int(lib().conv_bwd_weight_workspace_bytes(_pref(params)))


def conv_bwd_weight_bf16(params, x, dout, dw, db, ws, ws_bytes, stream=None):
    return lib().conv_bwd_weight_bf16(_pref(params), x, dout, dw, db, ws, ws_bytes, stream)


def _oref(opts):
    return None if opts is None else ctypes.byref(opts)


def conv_fwd_ex_workspace_bytes(params, opts, algo=0):
    return int(lib().conv_fwd_ex_workspace_bytes(_pref(params), _oref(opts), algo))


def conv_fwd_ex_bf16(params, opts, x, w, bias, y, ws, ws_bytes, algo=0, stream=None):
    return lib().conv_fwd_ex_bf16(_pref(params), _oref(opts), x, w, bias, y, ws, ws_bytes, algo, stream)


def conv_fwd_ex_f32(params, opts, x, w, bias, y, algo=0, stream=None):
    return lib().conv_fwd_ex_f32(_pref(params), _oref(opts), x, w, bias, y, algo, stream)


def conv_causal_fwd(seq, K, silu, x, ldx, w, bias, state, y, ldy, state_out, stream=None):
    return lib().conv_causal_fwd(_pref(seq), K, silu, x, ldx, w, bias, state, y, ldy, state_out, stream)


def conv_causal_bwd_workspace_bytes(seq, K):
    return int(lib().conv_causal_bwd_workspace_bytes(_pref(seq), K))


def conv_causal_bwd(seq, K, silu, x, ldx, w, bias, state, dy, lddy, dx, lddx, dw, db, dstate, ws, ws_bytes,
                    stream=None):
    return lib().conv_causal_bwd(_pref(seq), K, silu, x, ldx, w, bias, state, dy, lddy, dx, lddx, dw, db, dstate, ws,
                                 ws_bytes, stream)


def conv_causal_step(seq, K, silu, x, ldx, w, bias, state, y, ldy, stream=None):
    return lib().conv_causal_step(_pref(seq), K, silu, x, ldx, w, bias, state, y, ldy, stream)


def conv_scan_fwd_workspace_bytes(seq):
    return int(lib().conv_scan_fwd_workspace_bytes(_pref(seq)))


def conv_scan_fwd(seq, scale, x, ldx, gate, ldg, inp, ldi, decay, h0, y, ldy, hT, states, ws, ws_bytes, stream=None):
    return lib().conv_scan_fwd(_pref(seq), scale, x, ldx, gate, ldg, inp, ldi, decay, h0, y, ldy, hT, states, ws,
                               ws_bytes, stream)


def conv_scan_bwd_workspace_bytes(seq):
    return int(lib().conv_scan_bwd_workspace_bytes(_pref(seq)))


def conv_scan_bwd(seq, scale, x, ldx, gate, ldg, inp, ldi, decay, states, dy, lddy, dhT, dx, lddx, dgate, lddg, dinp,
                  lddi, ddecay, dh0, ws, ws_bytes, stream=None):
    return lib().conv_scan_bwd(_pref(seq), scale, x, ldx, gate, ldg, inp, ldi, decay, states, dy, lddy, dhT, dx, lddx,
                               dgate, lddg, dinp, lddi, ddecay, dh0, ws, ws_bytes, stream)


def conv_scan_step(seq, scale, x, ldx, gate, ldg, inp, ldi, decay, h, y, ldy, stream=None):
    return lib().conv_scan_step(_pref(seq), scale, x, ldx, gate, ldg, inp, ldi, decay, h, y, ldy, stream)


def conv_adamw_step(opt, tensors, count, stream=None):
    """tensors: a ctypes array of AdamwTensor (host memory), or None."""
    return lib().conv_adamw_step(_pref(opt), tensors, count, stream)


def conv_adamw_state_values(tensors, count, m_out, v_out, stream=None):
    """tensors as in conv_adamw_step; m_out, v_out: ctypes arrays of count device pointers."""
    return lib().conv_adamw_state_values(tensors, count, m_out, v_out, stream)


def make_params(x_shape, w_shape, stride=1, pad=0, dilation=1, groups=1):
    """ConvParams from NC(D)HW input and OI(D)HW weight shapes."""
    ndim = len(x_shape) - 2
    if ndim not in (2, 3) or len(w_shape) != ndim + 2:
        raise ValueError("expected 4-D or 5-D x and a weight of the same rank")
    sp = list(x_shape[2:])
    return ConvParams(ndim, x_shape[0], x_shape[1], sp[0] if ndim == 3 else 1, sp[-2], sp[-1], w_shape[0],
                      w_shape[2], stride, pad, dilation, groups)


# ---- torch-tensor helpers (device memory + stream plumbing only) --------------

_torch_module = None


def _torch():
    """torch, imported at the first call of a helper (the import statement itself takes 0.2 us each time)."""
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream():
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_tensor(t, name, dtypes):
    torch = _torch()
    if t is None:
        return
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous (NCHW / OIHW dense)" % name)
    _ = torch


def _dims(x, w, ndim):
    if x.dim() != ndim + 2 or w.dim() != ndim + 2:
        raise ValueError("expected %d-D x and w, got %s and %s" % (ndim + 2, tuple(x.shape), tuple(w.shape)))
    K = w.shape[2]
    if any(k != K for k in w.shape[2:]):
        raise ValueError("only square/cubic kernels are supported")
    if w.shape[1] != x.shape[1]:
        raise ValueError("w.shape[1]=%d != C_in=%d" % (w.shape[1], x.shape[1]))
    return K


def _out_shape(x, w, stride, pad, ndim):
    K = w.shape[2]
    outs = [conv_out_dim(d, K, stride, pad) for d in x.shape[2:]]
    return (x.shape[0], w.shape[0], *outs)


def workspace_for(x, w, stride=1, pad=0, algo="auto"):
    """A device workspace tensor sized for conv(..., workspace=...) (or None)."""
    torch = _torch()
    if x.dim() != 4 or x.dtype == torch.float32:
        return None
    a = ALGO[algo] if isinstance(algo, str) else int(algo)
    n = conv2d_fwd_workspace_bytes(x.shape[0], x.shape[1], x.shape[2], x.shape[3], w.shape[0],
                                   w.shape[2], stride, pad, a)
    return torch.empty(n, dtype=torch.uint8, device=x.device) if n else None


def conv(x, w, bias=None, stride=1, pad=0, algo="auto", out=None, workspace=None):
    """y = conv(x, w) + bias on the GPU.  x/w: bf16 (torch.bfloat16 or int16/uint16
    bit patterns) or float32, dense NC(D)HW / OI(D)HW; bias float32 or None.
    Returns float32 y.  2D or 3D by x.dim().  `workspace` (2D bf16 only, see
    workspace_for) selects conv2d_fwd_bf16_ws."""
    torch = _torch()
    ndim = x.dim() - 2
    if ndim not in (2, 3):
        raise ValueError("x must be 4-D (NCHW) or 5-D (NCDHW)")
    f32 = x.dtype == torch.float32
    half = (torch.bfloat16, torch.int16, torch.uint16)
    _check_tensor(x, "x", (torch.float32,) if f32 else half)
    _check_tensor(w, "w", (torch.float32,) if f32 else half)
    _check_tensor(bias, "bias", (torch.float32,))
    K = _dims(x, w, ndim)
    shape = _out_shape(x, w, stride, pad, ndim)
    if min(shape[2:]) < 1:
        raise ConvError(3, "conv")
    y = out if out is not None else torch.empty(shape, dtype=torch.float32, device=x.device)
    _check_tensor(y, "out", (torch.float32,))
    a = ALGO[algo] if isinstance(algo, str) else int(algo)
    args = [_ptr(x), _ptr(w), _ptr(bias), _ptr(y), x.shape[0], x.shape[1], *x.shape[2:],
            w.shape[0], K, stride, pad, a, _stream()]
    if ndim == 2 and workspace is not None and not f32:
        wsb = workspace.numel() * workspace.element_size()
        st = conv2d_fwd_bf16_ws(args[0], args[1], args[2], args[3], _ptr(workspace), wsb, *args[4:])
    elif ndim == 2:
        st = (conv2d_fwd_f32 if f32 else conv2d_fwd_bf16)(*args)
    else:
        st = (conv3d_fwd_f32 if f32 else conv3d_fwd_bf16)(*args)
    if st != CONV_OK:
        raise ConvError(st, "conv%dd_fwd" % ndim)
    return y


def pack_weights(w, x_shape, stride=1, pad=0, algo="auto", workspace=None):
    """Pack 2D bf16 weights for conv_prepacked (conv2d_pack_weights_bf16);
    returns the workspace tensor.  x_shape: (N, C_in, H, W) of the inputs the
    packed weights will be used with."""
    torch = _torch()
    _check_tensor(w, "w", (torch.bfloat16, torch.int16, torch.uint16))
    N, C, H, W = x_shape
    a = ALGO[algo] if isinstance(algo, str) else int(algo)
    need = conv2d_fwd_workspace_bytes(N, C, H, W, w.shape[0], w.shape[2], stride, pad, a)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=w.device)
    wsb = workspace.numel() * workspace.element_size()
    st = conv2d_pack_weights_bf16(_ptr(w), _ptr(workspace), wsb, N, C, H, W, w.shape[0], w.shape[2], stride,
                                  pad, a, _stream())
    if st != CONV_OK:
        raise ConvError(st, "conv2d_pack_weights_bf16")
    return workspace


def conv_prepacked(x, workspace, w_shape, bias=None, stride=1, pad=0, algo="auto", out=None):
    """conv(x, w) + bias with w taken from pack_weights' workspace (w_shape:
    the (C_out, C_in, K, K) shape of the packed weights)."""
    torch = _torch()
    _check_tensor(x, "x", (torch.bfloat16, torch.int16, torch.uint16))
    _check_tensor(bias, "bias", (torch.float32,))
    C_out, C_in, K = w_shape[0], w_shape[1], w_shape[2]
    if x.dim() != 4 or x.shape[1] != C_in:
        raise ValueError("x must be N x C_in x H x W with C_in = %d" % C_in)
    outs = [conv_out_dim(d, K, stride, pad) for d in x.shape[2:]]
    if min(outs) < 1:
        raise ConvError(3, "conv_prepacked")
    y = out if out is not None else torch.empty((x.shape[0], C_out, *outs), dtype=torch.float32,
                                                device=x.device)
    _check_tensor(y, "out", (torch.float32,))
    a = ALGO[algo] if isinstance(algo, str) else int(algo)
    wsb = workspace.numel() * workspace.element_size()
    st = conv2d_fwd_bf16_prepacked(_ptr(x), _ptr(workspace), wsb, _ptr(bias), _ptr(y), x.shape[0], C_in,
                                   x.shape[2], x.shape[3], C_out, K, stride, pad, a, _stream())
    if st != CONV_OK:
        raise ConvError(st, "conv2d_fwd_bf16_prepacked")
    return y


def im2col(x, K, stride=1, pad=0, out=None):
    """Explicit X_col (C_in*K^dims, N*prod(out)) as int16 bf16 bit patterns."""
    torch = _torch()
    ndim = x.dim() - 2
    _check_tensor(x, "x", (torch.bfloat16, torch.int16, torch.uint16))
    N, C = x.shape[:2]
    sp = list(x.shape[2:])
    D = sp[0] if ndim == 3 else 1
    nbytes = conv_im2col_bytes(ndim, N, C, D, sp[-2], sp[-1], K, stride, pad)
    if nbytes == 0:
        raise ConvError(2, "conv_im2col_bytes")
    outs = [conv_out_dim(d, K, stride, pad) for d in sp]
    cols = N
    for o in outs:
        cols *= o
    rows = C * K ** ndim
    col = out if out is not None else torch.empty((rows, cols), dtype=torch.int16, device=x.device)
    if ndim == 2:
        st = conv2d_im2col_bf16(_ptr(x), _ptr(col), N, C, sp[0], sp[1], K, stride, pad, _stream())
    else:
        st = conv3d_im2col_bf16(_ptr(x), _ptr(col), N, C, D, sp[1], sp[2], K, stride, pad, _stream())
    if st != CONV_OK:
        raise ConvError(st, "conv%dd_im2col_bf16" % ndim)
    return col


def conv_explicit(x, w, bias=None, stride=1, pad=0, workspace=None, out=None):
    """im2col into a workspace, then the MFMA GEMM; returns float32 y."""
    torch = _torch()
    ndim = x.dim() - 2
    half = (torch.bfloat16, torch.int16, torch.uint16)
    _check_tensor(x, "x", half)
    _check_tensor(w, "w", half)
    _check_tensor(bias, "bias", (torch.float32,))
    K = _dims(x, w, ndim)
    N, C = x.shape[:2]
    sp = list(x.shape[2:])
    D = sp[0] if ndim == 3 else 1
    nbytes = conv_im2col_bytes(ndim, N, C, D, sp[-2], sp[-1], K, stride, pad)
    if nbytes == 0:
        raise ConvError(2, "conv_im2col_bytes")
    ws = workspace if workspace is not None else torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    shape = _out_shape(x, w, stride, pad, ndim)
    y = out if out is not None else torch.empty(shape, dtype=torch.float32, device=x.device)
    wsb = ws.numel() * ws.element_size()
    if ndim == 2:
        st = conv2d_fwd_bf16_explicit(_ptr(x), _ptr(w), _ptr(bias), _ptr(y), _ptr(ws), wsb, N, C,
                                      sp[0], sp[1], w.shape[0], K, stride, pad, _stream())
    else:
        st = conv3d_fwd_bf16_explicit(_ptr(x), _ptr(w), _ptr(bias), _ptr(y), _ptr(ws), wsb, N, C,
                                      D, sp[1], sp[2], w.shape[0], K, stride, pad, _stream())
    if st != CONV_OK:
        raise ConvError(st, "conv%dd_fwd_bf16_explicit" % ndim)
    return y


def _general_out_shape(x, w, stride, pad, dilation):
    K = w.shape[2]
    outs = [conv_out_dim_dilated(d, K, stride, pad, dilation) for d in x.shape[2:]]
    return (x.shape[0], w.shape[0], *outs)


def _general_check(x, w, groups, half_ok=True):
    torch = _torch()
    ndim = x.dim() - 2
    if ndim not in (2, 3) or w.dim() != x.dim():
        raise ValueError("x must be 4-D or 5-D and w of the same rank")
    if any(k != w.shape[2] for k in w.shape[2:]):
        raise ValueError("only square/cubic kernels are supported")
    if groups < 1 or x.shape[1] % groups or w.shape[0] % groups or w.shape[1] * groups != x.shape[1]:
        raise ValueError("w.shape[1]=%d * groups=%d must equal C_in=%d and groups must divide C_out=%d"
                         % (w.shape[1], groups, x.shape[1], w.shape[0]))
    _ = torch
    return ndim


def conv_general(x, w, bias=None, stride=1, pad=0, dilation=1, groups=1, algo="auto", out=None):
    """y = conv(x, w) + bias with dilation and groups (conv_fwd_bf16 /
    conv_fwd_f32).  w: (C_out, C_in/groups, K, K[, K]).  Returns float32 y."""
    torch = _torch()
    _general_check(x, w, groups)
    f32 = x.dtype == torch.float32
    half = (torch.bfloat16, torch.int16, torch.uint16)
    _check_tensor(x, "x", (torch.float32,) if f32 else half)
    _check_tensor(w, "w", (torch.float32,) if f32 else half)
    _check_tensor(bias, "bias", (torch.float32,))
    shape = _general_out_shape(x, w, stride, pad, dilation)
    if min(shape[2:]) < 1:
        raise ConvError(3, "conv_general")
    y = out if out is not None else torch.empty(shape, dtype=torch.float32, device=x.device)
    _check_tensor(y, "out", (torch.float32,))
    prm = make_params(tuple(x.shape), tuple(w.shape), stride, pad, dilation, groups)
    a = ALGO[algo] if isinstance(algo, str) else int(algo)
    fn = conv_fwd_f32 if f32 else conv_fwd_bf16
    st = fn(prm, _ptr(x), _ptr(w), _ptr(bias), _ptr(y), a, _stream())
    if st != CONV_OK:
        raise ConvError(st, "conv_fwd_f32" if f32 else "conv_fwd_bf16")
    return y


def im2col_general(x, K, stride=1, pad=0, dilation=1, out=None):
    """X_col with dilated taps (conv_im2col_bf16) as int16 bf16 bit patterns."""
    torch = _torch()
    _check_tensor(x, "x", (torch.bfloat16, torch.int16, torch.uint16))
    ndim = x.dim() - 2
    prm = make_params(tuple(x.shape), (1, x.shape[1]) + (K,) * ndim, stride, pad, dilation, 1)
    nbytes = conv_xcol_bytes(prm)
    if nbytes == 0:
        raise ConvError(2, "conv_xcol_bytes")
    rows = x.shape[1] * K ** ndim
    col = out if out is not None else torch.empty((rows, nbytes // 2 // rows), dtype=torch.int16,
                                                  device=x.device)
    st = conv_im2col_bf16(prm, _ptr(x), _ptr(col), _stream())
    if st != CONV_OK:
        raise ConvError(st, "conv_im2col_bf16")
    return col


def conv_explicit_general(x, w, bias=None, stride=1, pad=0, dilation=1, groups=1, workspace=None, out=None):
    """conv_fwd_explicit_bf16: dilated im2col into a workspace, then one GEMM per group."""
    torch = _torch()
    _general_check(x, w, groups)
    half = (torch.bfloat16, torch.int16, torch.uint16)
    _check_tensor(x, "x", half)
    _check_tensor(w, "w", half)
    _check_tensor(bias, "bias", (torch.float32,))
    prm = make_params(tuple(x.shape), tuple(w.shape), stride, pad, dilation, groups)
    nbytes = conv_xcol_bytes(prm)
    if nbytes == 0:
        raise ConvError(2, "conv_xcol_bytes")
    ws = workspace if workspace is not None else torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    shape = _general_out_shape(x, w, stride, pad, dilation)
    y = out if out is not None else torch.empty(shape, dtype=torch.float32, device=x.device)
    st = conv_fwd_explicit_bf16(prm, _ptr(x), _ptr(w), _ptr(bias), _ptr(y), _ptr(ws),
                                ws.numel() * ws.element_size(), _stream())
    if st != CONV_OK:
        raise ConvError(st, "conv_fwd_explicit_bf16")
    return y


def conv_backward(x, w, dout, stride=1, pad=0, dilation=1, groups=1, with_db=True, out=None):
    """(dx, dw, db) of y = conv(x, w) + b for upstream gradient dout, all bf16
    inputs (conv_bwd_data_bf16 + conv_bwd_weight_bf16); fp32 results.  `out`:
    optional (dx, dw, db) tensors to write into."""
    torch = _torch()
    _general_check(x, w, groups)
    half = (torch.bfloat16, torch.int16, torch.uint16)
    for t, n in ((x, "x"), (w, "w"), (dout, "dout")):
        _check_tensor(t, n, half)
    prm = make_params(tuple(x.shape), tuple(w.shape), stride, pad, dilation, groups)
    yshape = _general_out_shape(x, w, stride, pad, dilation)
    if tuple(dout.shape) != tuple(yshape):
        raise ValueError("dout has shape %s, the output is %s" % (tuple(dout.shape), yshape))
    if out is None:
        dx = torch.empty(x.shape, dtype=torch.float32, device=x.device)
        dw = torch.empty(w.shape, dtype=torch.float32, device=x.device)
        db = torch.empty((w.shape[0],), dtype=torch.float32, device=x.device) if with_db else None
    else:
        dx, dw, db = out
    nd, nw = conv_bwd_data_workspace_bytes(prm), conv_bwd_weight_workspace_bytes(prm)
    wsd = torch.empty(max(nd, 16), dtype=torch.uint8, device=x.device)
    wsw = torch.empty(max(nw, 16), dtype=torch.uint8, device=x.device)
    st = conv_bwd_data_bf16(prm, _ptr(dout), _ptr(w), _ptr(dx), _ptr(wsd), wsd.numel(), _stream())
    if st != CONV_OK:
        raise ConvError(st, "conv_bwd_data_bf16")
    st = conv_bwd_weight_bf16(prm, _ptr(x), _ptr(dout), _ptr(dw), _ptr(db), _ptr(wsw), wsw.numel(), _stream())
    if st != CONV_OK:
        raise ConvError(st, "conv_bwd_weight_bf16")
    return dx, dw, db


def conv_ex(x, w, bias=None, stride=1, pad=0, dilation=1, groups=1, layout="nchw", out_dtype="f32", relu=False,
            algo="auto", workspace=None, out=None):
    """conv_fwd_ex_bf16 / conv_fwd_ex_f32.  layout "nhwc": x is (N, [D,] H, W, C)
    and y comes back (N, [D,] H, W, C_out); w stays (C_out, C_in/groups, K...).
    out_dtype "bf16": y holds bf16 bits (int16).  workspace: a tensor from
    workspace_ex() (packed 3x3 weights) or None."""
    torch = _torch()
    f32 = x.dtype == torch.float32
    half = (torch.bfloat16, torch.int16, torch.uint16)
    _check_tensor(x, "x", (torch.float32,) if f32 else half)
    _check_tensor(w, "w", (torch.float32,) if f32 else half)
    _check_tensor(bias, "bias", (torch.float32,))
    if layout == "nhwc":
        logical = (x.shape[0], x.shape[-1]) + tuple(x.shape[1:-1])
    else:
        logical = tuple(x.shape)
    prm = make_params(logical, tuple(w.shape), stride, pad, dilation, groups)
    opts = ConvOptions(LAYOUT[layout], OUT_DTYPE[out_dtype], int(bool(relu)))
    K = w.shape[2]
    outs = [conv_out_dim_dilated(d, K, stride, pad, dilation) for d in logical[2:]]
    if min(outs) < 1:
        raise ConvError(3, "conv_ex")
    shape = (logical[0], *outs, w.shape[0]) if layout == "nhwc" else (logical[0], w.shape[0], *outs)
    dt = torch.float32 if out_dtype == "f32" else torch.int16
    y = out if out is not None else torch.empty(shape, dtype=dt, device=x.device)
    a = ALGO[algo] if isinstance(algo, str) else int(algo)
    if f32:
        st = conv_fwd_ex_f32(prm, opts, _ptr(x), _ptr(w), _ptr(bias), _ptr(y), a, _stream())
    else:
        wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
        st = conv_fwd_ex_bf16(prm, opts, _ptr(x), _ptr(w), _ptr(bias), _ptr(y), _ptr(workspace), wsb, a, _stream())
    if st != CONV_OK:
        raise ConvError(st, "conv_fwd_ex")
    return y


def workspace_ex(x_shape, w_shape, stride=1, pad=0, dilation=1, groups=1, layout="nchw", out_dtype="f32",
                 relu=False, algo="auto", device="cuda"):
    """Workspace tensor for conv_ex (None when no route uses one); x_shape logical NC(D)HW."""
    torch = _torch()
    prm = make_params(tuple(x_shape), tuple(w_shape), stride, pad, dilation, groups)
    opts = ConvOptions(LAYOUT[layout], OUT_DTYPE[out_dtype], int(bool(relu)))
    a = ALGO[algo] if isinstance(algo, str) else int(algo)
    n = conv_fwd_ex_workspace_bytes(prm, opts, a)
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


# ---- sequences of tokens ------------------------------------------------------

_queries = None     # the current device, and the stream of a device, as integers


def _stream_of(t):
    """The current stream of t's device, which has to be the current one: the default stream of every device is
    the same null handle, which a launch takes as the current device's.  These helpers run once per token of
    an answer: the direct queries take 0.1 us, torch.cuda.current_stream_of(x) 3 us."""
    global _queries
    if _queries is None:
        torch = _torch()
        _queries = (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
                    getattr(torch._C, "_cuda_getCurrentRawStream", lambda d: torch.cuda.current_stream(d).cuda_stream))
    device, now = t.get_device(), _queries[0]()
    if device != now:
        raise ValueError("the tensors are on GPU %d, the current device is %d" % (device, now))
    return _queries[1](device)


def _dtype_code(t, name):
    """CONV_OUT_* of a float32 or bf16 (torch.bfloat16, or int16/uint16 bits) tensor."""
    torch = _torch()
    if t.dtype == torch.bfloat16:
        return 1
    if t.dtype == torch.float32:
        return 0
    if t.dtype in (torch.int16, torch.uint16):
        return 1
    raise TypeError("%s has dtype %s, expected float32 or bf16" % (name, t.dtype))


def _ld(t, shape, like, name, device=None):
    """The row stride of a tensor of rows: its last axis is dense, and its leading axes are one
    evenly strided axis (a column slice of a dense tensor, for instance)."""
    if t is like:
        if not t.is_cuda:
            raise ValueError("%s must be a GPU tensor" % name)
    else:
        if t.get_device() != (like.get_device() if device is None else device):
            raise ValueError("%s must be on x's GPU" % name)
        if t.shape != shape:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
        if t.dtype != like.dtype:
            raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, like.dtype))
    if t.is_contiguous():
        return shape[-1]
    if t.numel() == 0:
        return shape[-1]
    st = t.stride()
    if shape[-1] > 1 and st[-1] != 1:
        raise ValueError("%s: the channels of a row must be adjacent" % name)
    if len(shape) == 2:
        ld = st[0] if shape[0] > 1 else shape[1]
    elif shape[1] > 1:
        ld = st[1]
        if shape[0] > 1 and st[0] != shape[1] * ld:
            raise ValueError("%s: sequences must follow each other at the row stride" % name)
    else:
        ld = st[0] if shape[0] > 1 else shape[2]
    if ld < shape[-1]:
        raise ValueError("%s: rows overlap" % name)
    return ld


def _dense(t, shape, dtype, name, device):
    """The address of a dense tensor on x's GPU, `device`."""
    if t is None:
        return None
    if t.get_device() != device:
        raise ValueError("%s must be on x's GPU" % name)
    if t.dtype != dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


SEQ_FILL = 256      # CONV_SEQ_FILL


def make_seq(x, offsets=None, max_len=None, name="x", fill=False):
    """SeqParams for x: (B, T, C), or (tokens, C) packed, with offsets (B+1 int32 on the GPU) and
    max_len, the length of the longest sequence: a sequence's rows past it belong to none.  fill: rows of
    outputs that no sequence holds are set to zero (packed rows only; otherwise they are left)."""
    torch = _torch()
    code = _dtype_code(x, name)
    if offsets is None:
        if x.dim() != 3:
            raise ValueError("%s must be (sequences, tokens, channels), or packed rows with offsets" % name)
        return SeqParams(code, x.shape[0], x.shape[1], x.shape[2], None, 0)
    if x.dim() != 2:
        raise ValueError("packed %s must be (tokens, channels)" % name)
    if max_len is None:
        raise ValueError("packed sequences need max_len")
    if not offsets.is_cuda or offsets.dtype != torch.int32 or offsets.dim() != 1 or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int32 vector on the GPU")
    if offsets.get_device() != x.get_device():
        raise ValueError("offsets must be on the GPU of %s" % name)
    if offsets.shape[0] < 2:
        raise ValueError("offsets must hold B + 1 >= 2 values")
    return SeqParams(code + SEQ_FILL if fill else code, offsets.shape[0] - 1, max_len, x.shape[1], offsets.data_ptr(), x.shape[0])


def _step_seq(x):
    if x.dim() != 2:
        raise ValueError("x must be (sequences, channels)")
    return SeqParams(_dtype_code(x, "x"), x.shape[0], 1, x.shape[1], None, 0)


def _run(st, where):
    if st != CONV_OK:
        raise ConvError(st, where)


def _workspace(ws, need, x):
    """(address, bytes) of the workspace: the caller's, which the library holds to the size it needs, or a
    new one (returned too, to be kept for the call)."""
    torch = _torch()
    if ws is None:
        if not need:
            return None, 0, None
        ws = torch.empty(need, dtype=torch.uint8, device=x.device)
    elif ws.get_device() != x.get_device() or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on x's GPU")
    return ws.data_ptr(), ws.numel() * ws.element_size(), ws


def _rows_out(out, x, name, fill=True):
    """An output of rows and its row stride.  fill: rows that no sequence holds are set by the call."""
    torch = _torch()
    if out is None and not fill:
        return torch.zeros(x.shape, dtype=x.dtype, device=x.device), x.shape[-1]
    if out is None:
        y = torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        return y, x.shape[-1]
    return out, _ld(out, x.shape, x, name)


def causal_conv(x, w, bias=None, silu=False, state=None, offsets=None, max_len=None, with_state=False, out=None):
    """Causal depthwise convolution over the tokens of x, (B, T, C) or packed (see make_seq), float32 or
    bf16: conv_causal_fwd.  w: (C, K) of x's dtype, tap K-1 on the token itself; bias: float32 (C);
    state: the K-1 rows before each sequence, (B, K-1, C) of x's dtype, or None for zeros.  x and out
    may be column slices of a wider tensor.  Packed rows that no sequence holds (in front of offsets[0],
    behind offsets[-1], past max_len) come back as zeros; in a given out they stay as they are.
    Returns y, or (y, state after the last tokens)."""
    torch = _torch()
    seq = make_seq(x, offsets, max_len, fill=out is None)
    dev = x.get_device()
    ldx = _ld(x, x.shape, x, "x")
    if w.dim() != 2:
        raise ValueError("w must be (channels, taps)")
    K = w.shape[1]
    rows = (seq.B, K - 1, seq.C)
    y, ldy = _rows_out(out, x, "out")
    end = torch.empty(rows, dtype=x.dtype, device=x.device) if with_state else None
    _run(conv_causal_fwd(seq, K, int(bool(silu)), x.data_ptr(), ldx, _dense(w, (seq.C, K), x.dtype, "w", dev),
                         _dense(bias, (seq.C,), torch.float32, "bias", dev), _dense(state, rows, x.dtype, "state", dev),
                         y.data_ptr(), ldy, end.data_ptr() if with_state else None, _stream_of(x)), "conv_causal_fwd")
    return (y, end) if with_state else y


def causal_conv_backward(x, w, dy, bias=None, silu=False, state=None, offsets=None, max_len=None, out=None):
    """(dx, dw, db, dstate) of y = causal_conv(x, w, bias, silu, state) for upstream gradient dy
    (conv_causal_bwd): dx and dstate of x's dtype, dw (C, K) and db (C) float32; dstate is None without
    a state.  `out`: dx to write into, perhaps a column slice.  Rows that no sequence holds: as in causal_conv."""
    torch = _torch()
    seq = make_seq(x, offsets, max_len, fill=out is None)
    dev = x.get_device()
    ldx, lddy = _ld(x, x.shape, x, "x"), _ld(dy, x.shape, x, "dy", dev)
    if w.dim() != 2:
        raise ValueError("w must be (channels, taps)")
    K = w.shape[1]
    rows = (seq.B, K - 1, seq.C)
    dx, lddx = _rows_out(out, x, "out")
    dw = torch.empty((seq.C, K), dtype=torch.float32, device=x.device)
    db = torch.empty((seq.C,), dtype=torch.float32, device=x.device)
    ds = torch.empty(rows, dtype=x.dtype, device=x.device) if state is not None else None
    n = conv_causal_bwd_workspace_bytes(seq, K)
    ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    _run(conv_causal_bwd(seq, K, int(bool(silu)), x.data_ptr(), ldx, _dense(w, (seq.C, K), x.dtype, "w", dev),
                         _dense(bias, (seq.C,), torch.float32, "bias", dev), _dense(state, rows, x.dtype, "state", dev),
                         dy.data_ptr(), lddy, dx.data_ptr(), lddx, dw.data_ptr(), db.data_ptr(),
                         None if ds is None else ds.data_ptr(), ws.data_ptr(), n, _stream_of(x)), "conv_causal_bwd")
    return dx, dw, db, ds


def causal_conv_step(x, w, state, bias=None, silu=False, out=None):
    """One new token, x (B, C), of each of B sequences: returns y (B, C) and moves state (B, K-1, C) on
    by the token in place (conv_causal_step)."""
    torch = _torch()
    seq = _step_seq(x)
    dev = x.get_device()
    ldx = _ld(x, x.shape, x, "x")
    if w.dim() != 2:
        raise ValueError("w must be (channels, taps)")
    K = w.shape[1]
    y, ldy = _rows_out(out, x, "out")
    _run(conv_causal_step(seq, K, int(bool(silu)), x.data_ptr(), ldx, _dense(w, (seq.C, K), x.dtype, "w", dev),
                          _dense(bias, (seq.C,), torch.float32, "bias", dev),
                          _dense(state, (seq.B, K - 1, seq.C), x.dtype, "state", dev), y.data_ptr(), ldy, _stream_of(x)),
         "conv_causal_step")
    return y


SCAN_BLOCK = 64     # CONV_SCAN_BLOCK


def gated_scan(x, gate, inp, decay, scale=8.0, h0=None, offsets=None, max_len=None, with_states=False, out=None,
               workspace=None):
    """The gated linear recurrence over the tokens of x, (B, T, C) or packed (see make_seq), float32 or
    bf16 (conv_scan_fwd):

        a = exp(-scale * softplus(decay) * sigmoid(gate)),  h = a h + sqrt(1 - a^2) sigmoid(inp) x

    gate and inp: like x; decay: float32 (C); h0: float32 (B, C) or None for zeros.  x, gate, inp and out
    may be column slices of wider tensors.  workspace: a uint8 tensor of
    conv_scan_fwd_workspace_bytes(make_seq(x, ...)) bytes to use, or None to allocate one.  Packed rows that
    no sequence holds (in front of offsets[0], behind offsets[-1], past max_len) come back as zeros; in a given out they
    stay as they are.  Returns (y, h after the last tokens), and with_states also the states that gated_scan_backward
    starts from: float32 (B, ceil(T / 64), C), T being max_len for packed rows, not written past a sequence's end."""
    torch = _torch()
    seq = make_seq(x, offsets, max_len, fill=out is None)
    dev = x.get_device()
    ldx, ldg, ldi = _ld(x, x.shape, x, "x"), _ld(gate, x.shape, x, "gate", dev), _ld(inp, x.shape, x, "inp", dev)
    y, ldy = _rows_out(out, x, "out")
    ends = (seq.B, seq.C)
    hT = torch.empty(ends, dtype=torch.float32, device=x.device)
    states = None
    if with_states:
        states = torch.empty((seq.B, -(-seq.T // SCAN_BLOCK), seq.C), dtype=torch.float32, device=x.device)
    ws, wsb, held = _workspace(workspace, conv_scan_fwd_workspace_bytes(seq) if workspace is None else 0, x)
    _run(conv_scan_fwd(seq, scale, x.data_ptr(), ldx, gate.data_ptr(), ldg, inp.data_ptr(), ldi,
                       _dense(decay, (seq.C,), torch.float32, "decay", dev), _dense(h0, ends, torch.float32, "h0", dev),
                       y.data_ptr(), ldy, hT.data_ptr(), None if states is None else states.data_ptr(),
                       ws, wsb, _stream_of(x)), "conv_scan_fwd")
    return (y, hT, states) if with_states else (y, hT)


def gated_scan_backward(x, gate, inp, decay, dy, states, scale=8.0, dh=None, offsets=None, max_len=None, out=None,
                        workspace=None):
    """(dx, dgate, dinp, ddecay, dh0) of (y, h) = gated_scan(...) for upstream dy, like x, and dh, float32
    (B, C) or None for zeros (conv_scan_bwd).  states: as gated_scan(..., with_states=True) returned them
    for the same inputs.  `out`: (dx, dgate, dinp) to write into, perhaps column slices of one tensor, None for one to be
    allocated; rows that no sequence holds, and workspace (of conv_scan_bwd_workspace_bytes): as in gated_scan."""
    torch = _torch()
    seq = make_seq(x, offsets, max_len, fill=out is None)
    dev = x.get_device()
    ldx, ldg, ldi = _ld(x, x.shape, x, "x"), _ld(gate, x.shape, x, "gate", dev), _ld(inp, x.shape, x, "inp", dev)
    lddy = _ld(dy, x.shape, x, "dy", dev)
    o = (None, None, None) if out is None else out
    fill = out is None or offsets is None
    dx, lddx = _rows_out(o[0], x, "dx", fill)
    dg, lddg = _rows_out(o[1], x, "dgate", fill)
    di, lddi = _rows_out(o[2], x, "dinp", fill)
    ends = (seq.B, seq.C)
    dd = torch.empty((seq.C,), dtype=torch.float32, device=x.device)
    dh0 = torch.empty(ends, dtype=torch.float32, device=x.device)
    ws, wsb, held = _workspace(workspace, conv_scan_bwd_workspace_bytes(seq) if workspace is None else 0, x)
    nb = -(-seq.T // SCAN_BLOCK)
    _run(conv_scan_bwd(seq, scale, x.data_ptr(), ldx, gate.data_ptr(), ldg, inp.data_ptr(), ldi,
                       _dense(decay, (seq.C,), torch.float32, "decay", dev),
                       _dense(states, (seq.B, nb, seq.C), torch.float32, "states", dev), dy.data_ptr(), lddy,
                       _dense(dh, ends, torch.float32, "dh", dev), dx.data_ptr(), lddx, dg.data_ptr(), lddg, di.data_ptr(),
                       lddi, dd.data_ptr(), dh0.data_ptr(), ws, wsb, _stream_of(x)), "conv_scan_bwd")
    return dx, dg, di, dd, dh0


def gated_scan_step(x, gate, inp, decay, h, scale=8.0, out=None):
    """One new token, x, gate and inp (B, C), of each of B sequences: returns y (B, C) and updates h,
    float32 (B, C), in place (conv_scan_step)."""
    torch = _torch()
    seq = _step_seq(x)
    dev = x.get_device()
    ldx, ldg, ldi = _ld(x, x.shape, x, "x"), _ld(gate, x.shape, x, "gate", dev), _ld(inp, x.shape, x, "inp", dev)
    y, ldy = _rows_out(out, x, "out")
    _run(conv_scan_step(seq, scale, x.data_ptr(), ldx, gate.data_ptr(), ldg, inp.data_ptr(), ldi,
                        _dense(decay, (seq.C,), torch.float32, "decay", dev),
                        _dense(h, (seq.B, seq.C), torch.float32, "h", dev), y.data_ptr(), ldy, _stream_of(x)), "conv_scan_step")
    return y


# ---- the optimiser step --------------------------------------------------------

class AdamW:
    """AdamW over a list of tensors, one call per step (conv_adamw_step).

    params: float32 master weights, updated in place; grads: float32 or bf16, all alike; m, v: moments,
    float32, or with bits=8 int8 and uint8 codes, and then m_scale, v_scale, float32 of ceil(n/256).
    Moments that are not given start at zero.  copies: bf16 tensors that receive the updated weights
    (what the convolutions read), or None.  weight_decay: a number, or one for each tensor.  steps: how
    many were taken before.  grad_scale: a float32 scalar on the GPU that multiplies every gradient (a clipping
    factor, for instance), or None.  The tensors are kept and their addresses laid out once; step() may be
    given other gradients of the same sizes.  8-bit moments round at random, by seed and step; lr and seed may
    be changed between steps.  No two tensors may share memory.  A step captured in a graph repeats its own number,
    rates and random bits at every replay (conv_adamw_step): call step() beside the graph."""

    def __init__(self, params, grads, m=None, v=None, copies=None, bits=32, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
                 weight_decay=0.0, seed=0, steps=0, m_scale=None, v_scale=None, grad_scale=None):
        torch = _torch()
        if bits not in (8, 32):
            raise ValueError("bits must be 8 or 32")
        n = len(params)
        decays = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(d) for d in weight_decay]

        def fresh(sizes, dtype):
            return [torch.zeros(k, dtype=dtype, device=p.device) for k, p in zip(sizes, params)]

        sizes, blocks = [p.numel() for p in params], [-(-p.numel() // 256) for p in params]
        kinds = (torch.float32, torch.float32) if bits == 32 else (torch.int8, torch.uint8)
        self.params, self.copies, self.bits = list(params), copies, bits
        self.m = list(m) if m is not None else fresh(sizes, kinds[0])
        self.v = list(v) if v is not None else fresh(sizes, kinds[1])
        self.m_scale = self.v_scale = None
        if bits == 8:
            self.m_scale = list(m_scale) if m_scale is not None else fresh(blocks, torch.float32)
            self.v_scale = list(v_scale) if v_scale is not None else fresh(blocks, torch.float32)
        self.steps, self.lr, self.betas, self.eps, self.seed = int(steps), lr, betas, eps, seed
        for name, got in (("m", self.m), ("v", self.v), ("copies", copies), ("weight_decay", decays),
                          ("m_scale", self.m_scale), ("v_scale", self.v_scale)):
            if got is not None and len(got) != n:
                raise ValueError("%s: %d entries for %d tensors" % (name, len(got), n))

        device = params[0].get_device() if n else -1

        def addr(t, size, dtypes, name):
            if not t.is_cuda or not t.is_contiguous():
                raise ValueError("%s must be contiguous GPU tensors" % name)
            if t.get_device() != device:
                raise ValueError("%s must be on the first parameter's GPU" % name)
            if t.dtype not in dtypes:
                raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
            if t.numel() != size:
                raise ValueError("%s has %d elements, expected %d" % (name, t.numel(), size))
            return t.data_ptr()

        half = (torch.bfloat16, torch.int16, torch.uint16)
        f32 = (torch.float32,)
        self._addr, self._half = addr, half
        self._table = (AdamwTensor * max(n, 1))()
        for i, e in enumerate(self._table[:n]):
            e.n, e.weight_decay = sizes[i], decays[i]
            e.p = addr(params[i], sizes[i], f32, "params")
            e.m = addr(self.m[i], sizes[i], (kinds[0],), "m")
            e.v = addr(self.v[i], sizes[i], (kinds[1],), "v")
            if bits == 8:
                e.m_scale = addr(self.m_scale[i], blocks[i], f32, "m_scale")
                e.v_scale = addr(self.v_scale[i], blocks[i], f32, "v_scale")
            if copies is not None and copies[i] is not None:
                e.copy = addr(copies[i], sizes[i], half, "copies")
        if grad_scale is not None and n:
            addr(grad_scale, 1, f32, "grad_scale")
        self.grad_scale = grad_scale
        self._opt = AdamwOptions(bits=bits, grad_scale=None if grad_scale is None else grad_scale.data_ptr())
        self._set_grads(grads)

    def _set_grads(self, grads):
        """All of the list, or, where an entry is refused, nothing of it."""
        torch = _torch()
        grads = list(grads)
        if len(grads) != len(self.params):
            raise ValueError("grads: %d entries for %d tensors" % (len(grads), len(self.params)))
        f32 = not grads or grads[0].dtype == torch.float32
        kinds = (torch.float32,) if f32 else self._half
        addrs = [self._addr(g, p.numel(), kinds, "grads") for g, p in zip(grads, self.params)]
        self.grads = grads
        self._opt.grad_dtype = 0 if f32 else 1
        for e, a in zip(self._table, addrs):
            e.g = a

    def step(self, grads=None):
        """One step; lr and seed may be set between steps.  A step that raises leaves the gradients as they were."""
        o = self._opt
        o.lr, (o.beta1, o.beta2), o.eps, o.seed, o.step = self.lr, self.betas, self.eps, self.seed, self.steps + 1
        before = self.grads
        if grads is not None:
            self._set_grads(grads)
        if self.params:
            try:
                _run(conv_adamw_step(o, self._table, len(self.params), _stream_of(self.params[0])), "conv_adamw_step")
            except ConvError:
                if grads is not None:
                    self._set_grads(before)
                raise
        self.steps += 1

    def state_values(self, out=None):
        """The moments as float32, (list of m, list of v): with bits=8 the values their codes stand for
        (conv_adamw_state_values), written to `out`, two such lists, when given."""
        torch = _torch()
        n = len(self.params)
        if out is not None and [len(side) for side in out] != [n, n]:
            raise ValueError("out: lists of %s tensors for the m and v of %d" % ([len(side) for side in out], n))
        if self.bits == 32:
            if out is not None:
                for to, t in zip(list(out[0]) + list(out[1]), self.m + self.v):
                    to.copy_(t)
                return out
            return [t.clone() for t in self.m], [t.clone() for t in self.v]
        if out is None:
            out = tuple([torch.empty(p.numel(), dtype=torch.float32, device=p.device) for p in self.params]
                        for _ in range(2))
        ptrs = []
        for side in out:
            ptrs.append((ctypes.c_void_p * max(n, 1))(*[self._addr(t, p.numel(), (torch.float32,), "out")
                                                        for t, p in zip(side, self.params)]))
        if n:
            _run(conv_adamw_state_values(self._table, n, ptrs[0], ptrs[1], _stream_of(self.params[0])),
                 "conv_adamw_state_values")
        return out
