"""The 8-bit projections around a gated delta rule layer (C ABI in ``include/gdr_i8.h``).

    q8, s8, hidden = gdr.add_rmsnorm_i8(x, norm_w, residual=hidden)            # norm, codes, scales
    q, k, v, z = gdr.matmul_i8(q8, s8, w_in, w_in_scale, out=(2048, 2048, 4096, 4096))
    o, state = gdr.chunk_prefill(...)                                          # the delta rule
    q8, s8 = gdr.gated_rmsnorm_i8(o, z, head_norm_w)                           # codes for the way out
    y = gdr.matmul_i8(q8, s8, w_out, w_out_scale)

Activations and weights are int8 codes with an fp32 scale for each token and each output
channel; residual stream, gate and outputs are bf16 or fp32.  Forward only.

Work is enqueued on the current stream, or on ``stream`` (a torch stream or a handle), which the
caller orders after whatever made the inputs (and last used the outputs that are given); memory used
there is not reused before it is done.  Calls allocate nothing but the outputs that are not given,
of the memory of the stream that writes them, and can be captured into graphs.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import struct
import warnings

import torch

__all__ = ["add_rmsnorm_i8", "gated_rmsnorm_i8", "matmul_i8", "quantize_rows_i8", "NORM_MAX_COLS",
           "MATMUL_I8_MAX_K", "MATMUL_I8_MAX_OUT"]

NORM_MAX_COLS = 32768     # most values in one row of the norms
MATMUL_I8_MAX_K = 131071  # longest reduction of matmul_i8
MATMUL_I8_MAX_OUT = 8     # most separate outputs of one product
_VP = ctypes.c_void_p


class NormDims(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("heads", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("gate_dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32),
                ("eps", ctypes.c_float), ("x_stride", ctypes.c_int64), ("r_stride", ctypes.c_int64),
                ("out_stride", ctypes.c_int64)]


class MatmulDims(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int32), ("K", ctypes.c_int32), ("n_out", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("out_cols", ctypes.c_int32 * MATMUL_I8_MAX_OUT),
                ("out_stride", ctypes.c_int64 * MATMUL_I8_MAX_OUT), ("a_stride", ctypes.c_int64),
                ("w_stride", ctypes.c_int64)]


# The same layouts packed into bytes, which takes a fraction of the time of filling a Structure.
_NORM = struct.Struct("@6if3q")
_MATMUL = struct.Struct(f"@4i{MATMUL_I8_MAX_OUT}i{MATMUL_I8_MAX_OUT}q2q")
_PTRS = struct.Struct(f"@{MATMUL_I8_MAX_OUT}Q")
assert _NORM.size == ctypes.sizeof(NormDims) and _MATMUL.size == ctypes.sizeof(MatmulDims)

_CODE = {torch.bfloat16: 0, torch.float32: 1}
_F32, _I8 = torch.float32, torch.int8
# the current stream's handle without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_L = None


def bind(L):
    """Argument types of the entry points of gdr_i8.h on the loaded library."""
    L.gdr_add_rmsnorm_i8.restype = ctypes.c_int
    L.gdr_add_rmsnorm_i8.argtypes = [_VP] * 8
    L.gdr_gated_rmsnorm_i8.restype = ctypes.c_int
    L.gdr_gated_rmsnorm_i8.argtypes = [_VP] * 7
    L.gdr_matmul_i8.restype = ctypes.c_int
    L.gdr_matmul_i8.argtypes = [_VP] * 8


def _lib():
    global _L
    if _L is None:
        import gated_delta_rule_70_amd as gdr

        _L = gdr.lib()
    return _L


BINDING_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")
BINDING_VERSION = 1
_B = None


class _NoBinding:
    """In the extension's place where it is not built: every call goes through Python."""
    add_rmsnorm = gated_rmsnorm = matmul = staticmethod(lambda *a: None)


def _binding():
    """The extension that takes ordinary calls straight to the library (csrc/binding.cpp)."""
    global _B
    if _B is None:
        L = _lib()
        if not os.path.exists(BINDING_PATH):
            warnings.warn(f"{BINDING_PATH} is not built: calls of the 8-bit operators take 3 to 5 us longer", RuntimeWarning,
                          stacklevel=3)
            _B = _NoBinding
            return _B
        spec = importlib.util.spec_from_file_location("_binding", BINDING_PATH)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        if getattr(m, "VERSION", 0) != BINDING_VERSION:
            raise RuntimeError(f"{BINDING_PATH} is of another version; rebuild it")
        m.bind(*(ctypes.cast(f, _VP).value for f in (L.gdr_add_rmsnorm_i8, L.gdr_gated_rmsnorm_i8, L.gdr_matmul_i8)),
               _current_device, _raw_stream)
        _B = m
    return _B


def _fail(status):
    import gated_delta_rule_70_amd as gdr

    raise gdr.GdrError(status, _lib().gdr_status_str(status).decode())


def _code(t, name):
    c = _CODE.get(t.dtype)
    if c is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")
    return c


def _stream(stream, dev, names, tensors):
    """The stream's handle, once all tensors are known to be on the current GPU (``dev``: that of
    one of them)."""
    if dev >= 0 and dev == _current_device():
        for t in tensors:
            if t is not None and t.get_device() != dev:
                break
        else:
            here = _raw_stream(dev)
            if stream is None:
                return here
            there = _handle(stream)
            if there != here:  # the allocator must not hand the memory on before that stream is done
                s = _torch_stream(stream)
                for t in tensors:
                    if t is not None:
                        t.record_stream(s)
            return there
    for name, t in zip(names, tensors):
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor")
    at = torch.cuda.current_device()
    for name, t in zip(names, tensors):
        if t is not None and t.get_device() != at:
            raise ValueError(f"{name} is on GPU {t.get_device()}, the current one is {at}")


def _handle(stream):
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _torch_stream(stream):
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = _handle(stream)  # 0: the default stream, which ExternalStream takes for no handle at all
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _elsewhere(stream, t):
    """Whether ``stream`` is another one than the current stream of t's GPU."""
    return t.is_cuda and _handle(stream) != _raw_stream(t.get_device())


def _on(stream, call, *args):
    """``call(*args)``, which makes new outputs, with ``stream`` as the current one, so that they come
    from that stream's memory: what the allocator takes from the current stream's may still be in use
    by work queued there, which another stream does not wait for.  They are kept until the current
    stream, on which the caller will read them, is done too."""
    here, there = torch.cuda.current_stream(), _torch_stream(stream)
    torch.cuda.set_stream(there)
    try:
        outs = call(*args)
    finally:
        torch.cuda.set_stream(here)
    for group, user in ((args, there), ((outs,), here)):
        for t in group:
            for u in t if isinstance(t, (tuple, list)) else (t,):
                if isinstance(u, torch.Tensor):
                    u.record_stream(user)
    return outs


def _rows(t, name, tail=1):
    """Elements from one row to the next of ``t``, whose last ``tail`` dimensions make a row: a
    row's values have to lie next to each other, and the rows evenly apart."""
    shape, strides = t.shape, t.stride()
    lead = len(shape) - tail
    step = 1
    for i in range(len(shape) - 1, lead - 1, -1):
        if shape[i] != 1 and strides[i] != step:
            raise ValueError(f"{name}: the values of a row must be contiguous")
        step *= shape[i]
    row = None
    want = 0
    for i in range(lead - 1, -1, -1):
        if shape[i] == 1:
            continue
        if row is None:
            row = strides[i]
        elif strides[i] != want and t.numel():
            raise ValueError(f"{name}: rows must be evenly spaced")
        want = strides[i] * shape[i]
    return step if row is None or t.numel() == 0 else row


def _out(t, name, shape, dtype, device):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _eps(eps):
    raise ValueError(f"eps must be finite in fp32 and not negative, got {eps}")


_F32_MAX = 3.4028234663852886e38
_NORM_NAMES = ("weight", "residual", "q", "scale", "out_residual", "x")
_GATED_NAMES = ("gate", "weight", "q", "scale", "o")


def add_rmsnorm_i8(x, weight, residual=None, eps: float = 1e-6, q=None, scale=None, out_residual=None, stream=None):
    """Residual addition, root-mean-square norm, int8 codes (gdr_add_rmsnorm_i8).

    ``x`` and ``residual`` are ``[..., D]`` (bf16 or fp32, rows evenly spaced), ``weight`` ``[D]``
    (their type, or fp32).  With ``s = x + residual`` rounded to x's type, the norm of s times
    weight is returned as ``q`` (int8, ``[..., D]``) and ``scale`` (fp32, ``[...]``): it stands
    for ``q * scale[..., None]``.  Returns ``(q, scale, s)``; s is written to ``out_residual``
    (which may be ``x`` or ``residual`` itself), and is None without a residual.  A row of
    zeros has scale 0, a row that holds NaN or infinity scale NaN and q 0.
    """
    if stream is None:
        status = (_B or _binding()).add_rmsnorm(x, weight, residual, eps, q, scale, out_residual)
        if status is not None:
            if status:
                _fail(status)
            return q, scale, out_residual
    elif (q is None or scale is None or out_residual is None and residual is not None) and _elsewhere(stream, x):
        return _on(stream, add_rmsnorm_i8, x, weight, residual, eps, q, scale, out_residual)
    shape, dtype = x.shape, x.dtype
    if not shape or shape[-1] < 1:
        raise ValueError(f"x must be [..., D], got {list(shape)}")
    D = shape[-1]
    if D > NORM_MAX_COLS:
        raise ValueError(f"x has {D} values in a row, at most {NORM_MAX_COLS} are supported")
    xc = _code(x, "x")
    if weight.shape != (D,):
        raise ValueError(f"weight must be {[D]}, got {list(weight.shape)}")
    wt = weight.dtype
    if wt is not dtype and wt is not _F32:
        raise TypeError(f"weight must be {dtype} or float32, got {wt}")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    r_stride = out_stride = 0
    if residual is None:
        if out_residual is not None:
            raise ValueError("out_residual is given without a residual")
    else:
        if residual.shape != shape:
            raise ValueError(f"residual must be {list(shape)}, got {list(residual.shape)}")
        if residual.dtype is not dtype:
            raise TypeError(f"residual must be {dtype}, got {residual.dtype}")
        r_stride = D if residual.is_contiguous() else _rows(residual, "residual")
        if out_residual is None:
            out_residual = torch.empty(shape, dtype=dtype, device=x.device)
        if out_residual.shape != shape:
            raise ValueError(f"out_residual must be {list(shape)}, got {list(out_residual.shape)}")
        if out_residual.dtype is not dtype:
            raise TypeError(f"out_residual must be {dtype}, got {out_residual.dtype}")
        out_stride = D if out_residual.is_contiguous() else _rows(out_residual, "out_residual")
    lead = shape[:-1]
    if q is None or q.shape != shape or q.dtype is not _I8 or not q.is_contiguous():
        q = _out(q, "q", shape, _I8, x.device)
    if scale is None or scale.shape != lead or scale.dtype is not _F32 or not scale.is_contiguous():
        scale = _out(scale, "scale", lead, _F32, x.device)
    dims = _NORM.pack(scale.numel(), 1, D, xc, 0, _CODE[wt], eps if 0 <= eps <= _F32_MAX else _eps(eps),
                      D if x.is_contiguous() else _rows(x, "x"), r_stride, out_stride)
    s = _stream(stream, x.get_device(), _NORM_NAMES, (weight, residual, q, scale, out_residual, x))
    status = (_L or _lib()).gdr_add_rmsnorm_i8(
        dims, x.data_ptr(), None if residual is None else residual.data_ptr(), weight.data_ptr(), q.data_ptr(),
        scale.data_ptr(), None if out_residual is None else out_residual.data_ptr(), s)
    if status:
        _fail(status)
    return q, scale, out_residual


def gated_rmsnorm_i8(o, gate, weight, eps: float = 1e-6, q=None, scale=None, stream=None):
    """Norm of each value head of ``o``, times ``weight`` and silu(``gate``), as int8 codes with a
    scale for each token (gdr_gated_rmsnorm_i8).

    ``o`` and ``gate`` are ``[..., HV, dv]`` (bf16 or fp32 each; dv 32, 64 or 128), ``weight``
    ``[dv]`` (bf16 or fp32).  Returns ``q`` (int8, ``[..., HV * dv]``) and ``scale`` (fp32, ``[...]``).
    """
    if stream is None:
        status = (_B or _binding()).gated_rmsnorm(o, gate, weight, eps, q, scale)
        if status is not None:
            if status:
                _fail(status)
            return q, scale
    elif (q is None or scale is None) and _elsewhere(stream, o):
        return _on(stream, gated_rmsnorm_i8, o, gate, weight, eps, q, scale)
    shape = o.shape
    if len(shape) < 2:
        raise ValueError(f"o must be [..., HV, dv], got {list(shape)}")
    H, V = shape[-2:]
    if V not in (32, 64, 128):
        raise ValueError(f"dv must be 32, 64 or 128, got {V}")
    if H < 1 or H * V > NORM_MAX_COLS:
        raise ValueError(f"HV * dv must be in 1 .. {NORM_MAX_COLS}, got {H * V}")
    if gate.shape != shape:
        raise ValueError(f"gate must be {list(shape)}, got {list(gate.shape)}")
    if weight.shape != (V,):
        raise ValueError(f"weight must be {[V]}, got {list(weight.shape)}")
    oc, gc, wc = _code(o, "o"), _code(gate, "gate"), _code(weight, "weight")
    if not weight.is_contiguous():
        raise ValueError("weight must be contiguous")
    lead = shape[:-2]
    D = H * V
    qshape = (*lead, D)
    if q is None or q.shape != qshape or q.dtype is not _I8 or not q.is_contiguous():
        q = _out(q, "q", qshape, _I8, o.device)
    if scale is None or scale.shape != lead or scale.dtype is not _F32 or not scale.is_contiguous():
        scale = _out(scale, "scale", lead, _F32, o.device)
    dims = _NORM.pack(scale.numel(), H, V, oc, gc, wc, eps if 0 <= eps <= _F32_MAX else _eps(eps),
                      D if o.is_contiguous() else _rows(o, "o", 2),
                      D if gate.is_contiguous() else _rows(gate, "gate", 2), 0)
    s = _stream(stream, o.get_device(), _GATED_NAMES, (gate, weight, q, scale, o))
    status = (_L or _lib()).gdr_gated_rmsnorm_i8(dims, o.data_ptr(), gate.data_ptr(), weight.data_ptr(),
                                                 q.data_ptr(), scale.data_ptr(), s)
    if status:
        _fail(status)
    return q, scale


def matmul_i8(a, a_scale, w, w_scale, bias=None, out=None, out_dtype=torch.bfloat16, stream=None):
    """``(a @ w.T) * a_scale[..., None] * w_scale (+ bias)`` for int8 codes (gdr_matmul_i8).

    ``a`` is ``[..., K]`` and ``w`` ``[N, K]`` (int8, rows evenly spaced), ``a_scale`` ``[...]``,
    ``w_scale`` and ``bias`` ``[N]`` (fp32).  The sum is exact; ``out_dtype`` is bf16 or fp32.

    ``out`` says where the columns go: None for one new tensor ``[..., N]``, a tensor for one
    output, a sequence of column counts for that many new tensors, or a sequence of tensors (of
    one type; their rows may be strided).  Returns a tensor, or a tuple for a sequence.

    Fastest where rows of ``a`` and ``w`` begin at whole lines of 128 bytes: a reduction that is no
    multiple of 128 is better padded, codes of zero behind each row of both, or rows kept further
    apart (4096 x 4096 x 4097 takes half as long again as x 4096, x 4100 a quarter).
    """
    if stream is None:
        status = (_B or _binding()).matmul(a, a_scale, w, w_scale, bias, out)
        if status is not None:
            if status:
                _fail(status)
            return out if isinstance(out, torch.Tensor) else tuple(out)
    elif not isinstance(out, torch.Tensor) and _elsewhere(stream, a):
        return _on(stream, matmul_i8, a, a_scale, w, w_scale, bias, out, out_dtype)
    shape, wshape = a.shape, w.shape
    if not shape or len(wshape) != 2 or shape[-1] != wshape[1]:
        raise ValueError(f"a must be [..., K] and w [N, K], got {list(shape)} and {list(wshape)}")
    lead, (N, K) = shape[:-1], wshape
    if N < 1 or not 1 <= K <= MATMUL_I8_MAX_K:
        raise ValueError(f"N must be at least 1 and K in 1 .. {MATMUL_I8_MAX_K}, got N={N} K={K}")
    if a.dtype is not _I8:
        raise TypeError(f"a must be int8, got {a.dtype}")
    if w.dtype is not _I8:
        raise TypeError(f"w must be int8, got {w.dtype}")
    if a_scale is None or a_scale.shape != lead or a_scale.dtype is not _F32 or not a_scale.is_contiguous():
        _vector(a_scale, "a_scale", lead)
    if w_scale is None or w_scale.shape != (N,) or w_scale.dtype is not _F32 or not w_scale.is_contiguous():
        _vector(w_scale, "w_scale", (N,))
    if bias is not None:
        _vector(bias, "bias", (N,))
    single = out is None or isinstance(out, torch.Tensor)
    outs = [N] if out is None else [out] if single else list(out)
    n = len(outs)
    if not 1 <= n <= MATMUL_I8_MAX_OUT:
        raise ValueError(f"1 to {MATMUL_I8_MAX_OUT} outputs are supported, got {n}")
    for i, t in enumerate(outs):
        if isinstance(t, int) and t > 0:
            outs[i] = torch.empty(*lead, t, dtype=out_dtype, device=a.device)
    matrix = len(lead) == 1
    dtype, cols, strides, ptrs = None, [], [], []
    for t in outs:
        oshape = t.shape if isinstance(t, torch.Tensor) else ()
        if not oshape or oshape[-1] < 1:
            cols = [u.shape[-1] if isinstance(u, torch.Tensor) and u.dim() else u for u in outs]
            raise ValueError(f"the outputs' columns {cols} must be positive and add up to {N}")
        if (len(oshape) != 2 or oshape[0] != lead[0]) if matrix else oshape[:-1] != lead:
            raise ValueError(f"out must be {[*lead, oshape[-1]]}, got {list(oshape)}")
        if dtype is None:
            dtype, oc = t.dtype, _code(t, "out")
        elif t.dtype is not dtype:
            raise TypeError(f"outputs must be of one type, got {dtype} and {t.dtype}")
        cols.append(oshape[-1])
        strides.append(oshape[-1] if t.is_contiguous() else _rows(t, "out"))
        ptrs.append(t.data_ptr())
    if sum(cols) != N:
        raise ValueError(f"the outputs' columns {cols} must be positive and add up to {N}")
    none = _NONE[n:]
    dims = _MATMUL.pack(a_scale.numel(), K, n, oc, *cols, *none, *strides, *none,
                        K if a.is_contiguous() else _rows(a, "a"), K if w.is_contiguous() else _rows(w, "w"))
    s = _stream(stream, a.get_device(), _MATMUL_NAMES, (a, a_scale, w, w_scale, bias, *outs))
    status = (_L or _lib()).gdr_matmul_i8(dims, a.data_ptr(), a_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
                                          None if bias is None else bias.data_ptr(), _PTRS.pack(*ptrs, *none), s)
    if status:
        _fail(status)
    return outs[0] if single else tuple(outs)


_NONE = (0,) * MATMUL_I8_MAX_OUT
_MATMUL_NAMES = ("a", "a_scale", "w", "w_scale", "bias") + ("out",) * MATMUL_I8_MAX_OUT


def _vector(t, name, shape):
    if t is None:
        raise TypeError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.dtype is not _F32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def quantize_rows_i8(w):
    """int8 codes and fp32 scales of a weight matrix ``[N, K]``, a scale for each row (ties to
    even; a row of zeros has scale 0).  For preparing weights once; plain tensor operations on
    w's device.  Where K is no multiple of 128, columns of zeros behind w's and behind the
    activations' bring rows to whole lines (see matmul_i8)."""
    if w.dim() != 2 or not w.is_floating_point():
        raise ValueError(f"w must be a floating point matrix [N, K], got {list(w.shape)} {w.dtype}")
    top = w.double().abs().amax(1)
    codes = torch.round(w.double() * 127.0 / torch.where(top > 0, top, 1.0)[:, None])
    return codes.to(torch.int8), (top / 127.0).float()
