"""Python binding of include/svgemm_layer.h: the steps of a decoder layer around
the quantized linears.  Argument marshalling only, as in the package's main
module: every function checks devices, dtypes and shapes and calls the C entry
point of the same name on the current stream of the tensors' device (or the
stream given)."""
from __future__ import annotations

import ctypes

import torch

_FLOATS = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _bind(lib):
    vp, i, d = ctypes.c_void_p, ctypes.c_int, ctypes.c_double
    lib.add_rmsnorm_quant_i8.argtypes = [vp, i, vp, vp, i, d, i, i, vp, i, vp, vp, vp, vp]
    lib.add_rmsnorm_quant_i8.restype = ctypes.c_int


def _tensor(t, name, dtype, dev):
    """A contiguous tensor of dtype on dev: its address."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _float_tensor(t, name, dev):
    """As _tensor, of any of the element types: (address, type number)."""
    kind = _FLOATS.get(t.dtype)
    if kind is None:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {t.dtype}")
    return _tensor(t, name, t.dtype, dev), kind


def _device(t, name):
    dev = t.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a device tensor")
    return dev


def _call(fn, dev, stream, *args):
    """fn(*args, stream) with dev as the current device."""
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev.index)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if torch.cuda.current_device() == dev.index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        from . import SvgError, last_error
        raise SvgError(status, last_error())


def add_rmsnorm_quant_i8(x, residual, weight, eps, signs, xq, x_scale, y=None, block=32, stream=None):
    """residual += x (x alone without a residual), root-mean-square norm by
    weight, rotation and int8 quantization in one launch: x [M, K] fp32 / fp16
    / bf16, residual fp32 [M, K] or None, weight [K]; outputs xq (M * K codes,
    one slab buffer per 32 rows), x_scale [M] and, if given, the normalised
    rows y fp32 [M, K]."""
    dev = _device(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    px, kx = _float_tensor(x, "x", dev)
    pw, kw = _float_tensor(weight, "weight", dev)
    pr = None if residual is None else _tensor(residual, "residual", torch.float32, dev)
    py = None if y is None else _tensor(y, "y", torch.float32, dev)
    ps = _tensor(signs, "signs", torch.int8, dev)
    pq = _tensor(xq, "xq", torch.int8, dev)
    pc = _tensor(x_scale, "x_scale", torch.float32, dev)
    if ((residual is not None and residual.shape != x.shape) or (y is not None and y.shape != x.shape)
            or weight.numel() != K or signs.numel() != K or xq.numel() != M * K or x_scale.numel() != M):
        raise ValueError("need residual and y [M, K], weight and signs [K], xq of M * K codes and x_scale [M]")
    _call(_lib().add_rmsnorm_quant_i8, dev, stream, px, kx, pr, pw, kw, eps, M, K, ps, block, py, pq, pc)


def _lib():
    from . import lib
    return lib
