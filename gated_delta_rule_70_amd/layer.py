"""The operators in front of a recurrence and beside it (C ABI in ``include/gdr_layer.h``).

    q, k, v = gdr.matmul_i8(...)  or one tensor of all their columns
    (q, k, v), conv = gdr.causal_conv(qkv, conv_w, state=conv, out=(2048, 2048, 4096))
    q, k = gdr.qk_norm_rope(q, k, q_w, k_w, cos, sin)                     # norm per head, rotation
    o, state = gdr.chunk_prefill(q, k, v, ...)                             # the delta rule, or
    y, h = gdr.selective_scan(x, dt, A, B, C, D=D, z=z, dt_bias=bias, dt_softplus=True, h0=h)

and for one new token of each sequence, states updated in place:

    q, k, v = gdr.causal_conv_step(qkv, conv_w, conv, out=(2048, 2048, 4096))
    y = gdr.selective_scan_step(x, dt, A, B, C, h, D=D, z=z, dt_bias=bias, dt_softplus=True)

Activations are bf16 or fp32, sums and the scan's states fp32.  Forward only.  A batch is dense
(``[B, T, ...]``) or, with ``cu_seqlens`` (int32 ``[N + 1]`` on the GPU), N sequences laid end to end
(``[T, ...]``, or with a leading 1), as in ``chunk_prefill_varlen``: sequence i is on rows
``[cu_seqlens[i], cu_seqlens[i + 1])``, and rows outside all of them are not written.

Tensors may be strided where rows (tokens) are evenly spaced and a row's values contiguous: column
ranges of one projection's output, for instance.  Streams and the memory of new outputs as in
:mod:`.quantized`; calls allocate nothing but outputs that are not given, and the workspace of a
``selective_scan`` that needs one and is not given it, and can be captured.  A call with every tensor given goes
straight to the library (4 us from one to the next; others 10 to 19): of a scan that needs a workspace, that is
one with it.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import quantized as _qz
from .quantized import _code, _elsewhere, _eps, _fail, _on, _rows, _stream

__all__ = ["causal_conv", "causal_conv_step", "qk_norm_rope", "rope_table", "selective_scan", "selective_scan_step",
           "selective_scan_workspace_bytes", "CONV_MAX_OUT", "SCAN_MAX_STATES", "QK_MAX_DIM"]

CONV_MAX_OUT = 8        # most separate outputs of one convolution
SCAN_MAX_STATES = 128   # most state values of a channel
QK_MAX_DIM = 512        # most values of a head
MAX_ROWS = 1 << 30      # most rows (tokens) of one call
MAX_CHANNELS = 1 << 24
MAX_SEQS = 4096         # most sequences of a packed batch
_VP = ctypes.c_void_p
_F32 = torch.float32


class ConvDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "W", "dtype", "weight_dtype", "flags", "n_out")] + [
        ("out_cols", ctypes.c_int32 * CONV_MAX_OUT), ("out_stride", ctypes.c_int64 * CONV_MAX_OUT),
        ("x_stride", ctypes.c_int64)]


class QkDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("rows", "q_heads", "k_heads", "dim", "rotated", "table_rows", "period",
                                              "position_bits", "dtype", "weight_dtype", "flags")] + [
        ("eps", ctypes.c_float)] + [(n, ctypes.c_int64) for n in ("q_stride", "k_stride", "out_q_stride", "out_k_stride")]


class ScanDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "N", "G", "dtype", "dt_dtype", "flags")] + [
        (n, ctypes.c_int64) for n in ("x_stride", "dt_stride", "z_stride", "b_stride", "c_stride", "out_stride")]


# The same layouts packed into bytes, as in quantized.py.
_CONV = struct.Struct(f"@{8 + CONV_MAX_OUT}i{CONV_MAX_OUT + 1}q")
_QK = struct.Struct("@11if4q")
_SCAN = struct.Struct("@8i6q")
_PTRS = struct.Struct(f"@{CONV_MAX_OUT}Q")
assert (_CONV.size, _QK.size, _SCAN.size) == tuple(ctypes.sizeof(s) for s in (ConvDims, QkDims, ScanDims))
_NONE = (0,) * CONV_MAX_OUT


def bind(L):
    """Argument types of the entry points of gdr_layer.h on the loaded library."""
    for name, n in (("gdr_causal_conv", 9), ("gdr_qk_norm_rope", 11), ("gdr_selective_scan", 16),
                    ("gdr_selective_scan_step", 13)):
        fn = getattr(L, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.c_size_t if (name, i) == ("gdr_selective_scan", 14) else _VP for i in range(n)]
    L.gdr_selective_scan_workspace_bytes.restype = ctypes.c_size_t
    L.gdr_selective_scan_workspace_bytes.argtypes = [_VP, ctypes.c_int]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stride(t, name, tail=1):
    """Elements from one row of t to the next (a row: the last ``tail`` dimensions)."""
    if t.is_contiguous():
        n = 1
        for s in t.shape[len(t.shape) - tail:]:
            n *= s
        return n
    return _rows(t, name, tail)


def _need(t, name, shape, dtype, dense=True):
    """t is a tensor of this shape and type (one of the types given), contiguous if ``dense``."""
    if t is None:
        raise TypeError(f"{name} is required")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    types = dtype if isinstance(dtype, tuple) else (dtype,)
    if t.dtype not in types:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dict.fromkeys(types))}, got {t.dtype}")
    if dense and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _batch(x, cu_seqlens):
    """(sequences, T of the dims, leading shape) of x ``[B, T, D]``, or ``[T, D]`` / ``[1, T, D]`` packed."""
    shape = x.shape
    if len(shape) and not 1 <= shape[-1] <= MAX_CHANNELS:
        raise ValueError(f"x must have 1 to {MAX_CHANNELS} channels, got {list(shape)}")
    if cu_seqlens is None:
        if len(shape) != 3:
            raise ValueError(f"x must be [B, T, D], got {list(shape)}")
        B, T = shape[:2]
        rows = B * T
    else:
        if len(shape) not in (2, 3) or len(shape) == 3 and shape[0] != 1:
            raise ValueError(f"x must be [T, D] (or [1, T, D]) for a packed batch, got {list(shape)}")
        if cu_seqlens.dim() != 1 or not 2 <= cu_seqlens.shape[0] <= MAX_SEQS + 1:
            raise ValueError(f"cu_seqlens must be [N + 1] with N in 1 .. {MAX_SEQS}, got {list(cu_seqlens.shape)}")
        if cu_seqlens.dtype is not torch.int32:
            raise TypeError(f"cu_seqlens must be int32, got {cu_seqlens.dtype}")
        if not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous")
        B, T = cu_seqlens.shape[0] - 1, shape[-2]
        rows = T
    if max(rows, B, T) > MAX_ROWS:
        raise ValueError(f"x has {rows} rows in {B} sequences, at most {MAX_ROWS} are supported")
    return B, T, shape[:-1]


def _tokens(x):
    """The same of x ``[B, D]``, one token of each sequence."""
    if x.dim() != 2 or not 1 <= x.shape[1] <= MAX_CHANNELS:
        raise ValueError(f"x must be [B, D] with D in 1 .. {MAX_CHANNELS}, got {list(x.shape)}")
    if x.shape[0] > MAX_ROWS:
        raise ValueError(f"x has {x.shape[0]} rows, at most {MAX_ROWS} are supported")
    return x.shape[0], 1, x.shape[:1]


def causal_conv(x, weight, bias=None, state=None, cu_seqlens=None, activation="silu", out=None, out_state=None,
                want_state: bool = True, stream=None):
    """Short causal convolution of each channel over time (gdr_causal_conv).

    ``y[t] = act(bias + sum_j weight[:, j] * x[t - (W - 1) + j])``: ``x`` is ``[B, T, D]`` (bf16 or
    fp32), ``weight`` ``[D, W]`` (W 2 to 4; the last column is the current token's) and ``bias``
    ``[D]`` of x's type or fp32, ``state`` ``[B, W - 1, D]`` of x's type the rows before the first one,
    oldest first (None: zeros).  ``activation`` is "silu" or None.

    ``out`` says where the channels go, as in ``matmul_i8``: None for one new tensor, a tensor, a
    sequence of channel counts for that many new tensors, or a sequence of tensors.  Returns
    ``(y, out_state)``, y a tuple for a sequence; ``out_state`` (which may be ``state`` itself) holds
    the rows that a later call continues from, and is None if not given and not wanted.
    """
    if stream is None:
        status = (_qz._B or _qz._binding()).causal_conv(x, weight, bias, state, cu_seqlens, activation, out, out_state, want_state,
                                                        False)
        if status is not None:
            if status:
                _fail(status)
            return (out if isinstance(out, torch.Tensor) else tuple(out)), out_state
    else:
        out = _listed(out)
        if (not _given(out) or out_state is None and want_state) and _elsewhere(stream, x):
            return _on(stream, causal_conv, x, weight, bias, state, cu_seqlens, activation, out, out_state, want_state)
    return _conv(x, weight, bias, state, cu_seqlens, activation, out, out_state, want_state, stream,
                 *_batch(x, cu_seqlens))


def causal_conv_step(x, weight, state, bias=None, activation="silu", out=None, out_state=None, stream=None):
    """One new token of every sequence through :func:`causal_conv`: ``x`` is ``[B, D]``.  Updates
    ``state`` in place unless ``out_state`` is given.  Returns y (a tuple for a sequence ``out``).
    ``state`` may be None (zeros; ``out_state`` then receives the new state if given)."""
    end = state if out_state is None else out_state
    if stream is None:
        status = (_qz._B or _qz._binding()).causal_conv(x, weight, bias, state, None, activation, out, end, False, True)
        if status is not None:
            if status:
                _fail(status)
            return out if isinstance(out, torch.Tensor) else tuple(out)
    else:
        out = _listed(out)
        if not _given(out) and _elsewhere(stream, x):
            return _on(stream, causal_conv_step, x, weight, state, bias, activation, out, out_state)
    return _conv(x, weight, bias, state, None, activation, out, end, False, stream, *_tokens(x))[0]


def _listed(out):
    """``out`` as something that can be gone through more than once."""
    return out if out is None or isinstance(out, (torch.Tensor, tuple, list)) else list(out)


def _given(out):
    """Whether ``out`` leaves no tensor to be made."""
    return isinstance(out, torch.Tensor) or out is not None and all(isinstance(t, torch.Tensor) for t in out)


def _conv(x, weight, bias, state, cu, activation, out, out_state, want_state, stream, B, T, lead):
    D, dtype = x.shape[-1], x.dtype
    xc = _code(x, "x")
    if weight.dim() != 2 or weight.shape[0] != D or not 2 <= weight.shape[1] <= 4:
        raise ValueError(f"weight must be [{D}, W] with W in 2 .. 4, got {list(weight.shape)}")
    W = weight.shape[1]
    _need(weight, "weight", (D, W), (dtype, _F32))
    if bias is not None:
        _need(bias, "bias", (D,), weight.dtype)
    if activation not in ("silu", None):
        raise ValueError(f"activation must be 'silu' or None, got {activation!r}")
    if state is not None:
        _need(state, "state", (B, W - 1, D), dtype)
    if out_state is None and want_state:
        out_state = torch.empty((B, W - 1, D), dtype=dtype, device=x.device)
    if out_state is not None:
        _need(out_state, "out_state", (B, W - 1, D), dtype)
    single = out is None or isinstance(out, torch.Tensor)
    outs = [D] if out is None else [out] if single else list(out)
    n = len(outs)
    if not 1 <= n <= CONV_MAX_OUT:
        raise ValueError(f"1 to {CONV_MAX_OUT} outputs are supported, got {n}")
    for i, t in enumerate(outs):
        if isinstance(t, int) and t > 0:
            outs[i] = torch.empty(*lead, t, dtype=dtype, device=x.device)
    cols, strides = [], []
    for t in outs:
        if not isinstance(t, torch.Tensor) or not t.dim() or t.shape[-1] < 1:
            cols = [u.shape[-1] if isinstance(u, torch.Tensor) and u.dim() else u for u in outs]
            raise ValueError(f"the outputs' channels {cols} must be positive and add up to {D}")
        if t.shape[:-1] != lead:
            raise ValueError(f"out must be {[*lead, t.shape[-1]]}, got {list(t.shape)}")
        if t.dtype is not dtype:
            raise TypeError(f"out must be {dtype}, got {t.dtype}")
        cols.append(t.shape[-1])
        strides.append(_stride(t, "out"))
    if sum(cols) != D:
        raise ValueError(f"the outputs' channels {cols} must be positive and add up to {D}")
    none = _NONE[n:]
    dims = _CONV.pack(B, T, D, W, xc, _code(weight, "weight"), 1 if activation else 0, n, *cols, *none, *strides, *none,
                      _stride(x, "x"))
    s = _stream(stream, x.get_device(), _CONV_NAMES, (x, weight, bias, state, cu, out_state, *outs))
    status = _qz._lib().gdr_causal_conv(dims, _ptr(cu), x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(state),
                                        _PTRS.pack(*[t.data_ptr() for t in outs], *none), _ptr(out_state), s)
    if status:
        _fail(status)
    return (outs[0] if single else tuple(outs)), out_state


_CONV_NAMES = ("x", "weight", "bias", "state", "cu_seqlens", "out_state") + ("out",) * CONV_MAX_OUT


def rope_table(length, rotated, base: float = 10000.0, device=None):
    """``(cos, sin)`` for :func:`qk_norm_rope`: fp32 ``[length, rotated / 2]``, of the angles ``position *
    base ** (-2 i / rotated)``, computed in fp64.  For preparing them once; plain tensor operations."""
    if length < 1 or rotated < 2 or rotated % 2:
        raise ValueError(f"length must be positive and rotated even and positive, got {length} and {rotated}")
    speed = float(base) ** (-torch.arange(0, rotated, 2, device=device, dtype=torch.float64) / rotated)
    angle = torch.arange(length, device=device, dtype=torch.float64)[:, None] * speed
    return angle.cos().float(), angle.sin().float()


def qk_norm_rope(q, k, q_weight=None, k_weight=None, cos=None, sin=None, positions=None, eps: float = 1e-6,
                 interleaved: bool = False, out_q=None, out_k=None, stream=None):
    """Root-mean-square norm of each query and key head, then rotation by position (gdr_qk_norm_rope).

    ``q`` is ``[..., HQ, d]`` and ``k`` ``[..., HK, d]`` (bf16 or fp32, d at most 512), the weights
    ``[d]`` of their type or fp32 (None: ones), ``cos`` and ``sin`` fp32 ``[P, r / 2]`` (see
    :func:`rope_table`; None: no rotation).  The first r values of a head are rotated in pairs ``(i, i +
    r/2)``, or ``(2 i, 2 i + 1)`` if ``interleaved``.  ``positions`` (int32 or int64, ``[...]``) are rows of
    the tables; without them the position is the index along the last leading dimension.  The rotated
    values of a position outside the tables are NaN.

    The squared length instead of the mean (keys of length one): weights of ``d ** -0.5``, and eps / d.

    Returns ``(out_q, out_k)`` of q's and k's shapes; they may be ``q`` and ``k`` themselves.
    """
    if stream is None:
        status = (_qz._B or _qz._binding()).qk_norm_rope(q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, out_q, out_k)
        if status is not None:
            if status:
                _fail(status)
            return out_q, out_k
    elif (out_q is None or out_k is None) and _elsewhere(stream, q):
        return _on(stream, qk_norm_rope, q, k, q_weight, k_weight, cos, sin, positions, eps, interleaved, out_q, out_k)
    if q.dim() < 2 or k.dim() != q.dim() or k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
        raise ValueError(f"q must be [..., HQ, d] and k [..., HK, d], got {list(q.shape)} and {list(k.shape)}")
    lead, (HQ, d), HK, dtype = q.shape[:-2], q.shape[-2:], k.shape[-2], q.dtype
    if not 1 <= d <= QK_MAX_DIM or HQ < 1 or HK < 1:
        raise ValueError(f"d must be in 1 .. {QK_MAX_DIM} and heads positive, got {list(q.shape)} and {list(k.shape)}")
    qc = _code(q, "q")
    if k.dtype is not dtype:
        raise TypeError(f"k must be {dtype}, got {k.dtype}")
    wt = None
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _need(w, name, (d,), (dtype, _F32) if wt is None else wt)
            wt = w.dtype
    rows = 1
    for n in lead:
        rows *= n
    if rows > MAX_ROWS:
        raise ValueError(f"q has {rows} rows, at most {MAX_ROWS} are supported")
    rotated, length, period, bits = 0, 0, lead[-1] if lead else 1, 32
    if (cos is None) != (sin is None):
        raise TypeError("cos and sin are required together")
    if cos is not None:
        if cos.dim() != 2 or cos.shape[0] < 1 or not 1 <= cos.shape[1] <= d // 2:
            raise ValueError(f"cos must be [P, r / 2] with r at most {d}, got {list(cos.shape)}")
        _need(cos, "cos", cos.shape, _F32)
        _need(sin, "sin", cos.shape, _F32)
        length, rotated = cos.shape[0], 2 * cos.shape[1]
        if length > 2 ** 31 - 1:
            raise ValueError(f"cos has {length} rows, at most 2^31 - 1 are supported")
    if positions is not None:
        if cos is None:
            raise TypeError("positions are given without cos and sin")
        _need(positions, "positions", lead, (torch.int32, torch.int64))
        bits = 32 if positions.dtype is torch.int32 else 64
    out_q, out_k = (torch.empty(t.shape, dtype=dtype, device=t.device) if o is None else o for t, o in ((q, out_q), (k, out_k)))
    _need(out_q, "out_q", q.shape, dtype, dense=False)
    _need(out_k, "out_k", k.shape, dtype, dense=False)
    dims = _QK.pack(rows, HQ, HK, d, rotated, length, max(period, 1), bits, qc, qc if wt is None else _qz._CODE[wt],
                    1 if interleaved else 0, eps if 0 <= eps <= _qz._F32_MAX else _eps(eps), _stride(q, "q", 2),
                    _stride(k, "k", 2), _stride(out_q, "out_q", 2), _stride(out_k, "out_k", 2))
    s = _stream(stream, q.get_device(), _QK_NAMES, (q, k, q_weight, k_weight, cos, sin, positions, out_q, out_k))
    status = _qz._lib().gdr_qk_norm_rope(dims, q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(cos),
                                         _ptr(sin), _ptr(positions), out_q.data_ptr(), out_k.data_ptr(), s)
    if status:
        _fail(status)
    return out_q, out_k


_QK_NAMES = ("q", "k", "q_weight", "k_weight", "cos", "sin", "positions", "out_q", "out_k")


def selective_scan(x, dt, A, B, C, D=None, z=None, dt_bias=None, dt_softplus: bool = False, h0=None, cu_seqlens=None,
                   out=None, ht=None, want_state: bool = True, stream=None, workspace=None):
    """The recurrence with a diagonal, input-dependent transition over prompts (gdr_selective_scan).

    With ``step = dt + dt_bias`` (softplus of it with ``dt_softplus``), for every channel and its state
    ``h[N]``: ``h = exp(step * A) * h + step * x * B``; ``y = sum(C * h) + D * x``, times silu(``z``).

    ``x``, ``z`` are ``[B, T, D]`` (bf16 or fp32), ``dt`` ``[B, T, D]`` of x's type or fp32, ``B`` and ``C``
    ``[B, T, N]`` or ``[B, T, G, N]`` of x's type (groups of D / G channels share them; N at most 128),
    ``A`` ``[D, N]``, ``D`` and ``dt_bias`` ``[D]`` fp32, states ``[B, D, N]`` fp32.  Returns ``(y, ht)``, y of
    x's type; ``ht`` may be ``h0`` itself, and is None if not given and not wanted.

    Long sequences of few channels need a workspace (see :func:`selective_scan_workspace_bytes`), a contiguous
    uint8 tensor on x's GPU; one is allocated, in each call, if it is None.  Calls that overlap in time, or graphs
    replayed so, need one each.

    Infinite inputs and states give what the formula gives, but that what lies below fp32's normal range counts as
    zero: infinity times such a token's factor ``exp(step * A)``, or such a gate, is NaN.
    """
    if stream is None:
        status = (_qz._B or _qz._binding()).selective_scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, cu_seqlens, out, ht,
                                                           want_state, False, workspace)
        if status is not None:
            if status:
                _fail(status)
            return out, ht
    elif (out is None or ht is None and want_state) and _elsewhere(stream, x):
        return _on(stream, selective_scan, x, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, cu_seqlens, out, ht, want_state,
                   None, workspace)
    return _scan("gdr_selective_scan", x, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, cu_seqlens, out, ht, want_state,
                 stream, workspace, *_batch(x, cu_seqlens))


def selective_scan_workspace_bytes(B, T, D, N, groups: int = 1, packed: bool = False) -> int:
    """Bytes of workspace that :func:`selective_scan` needs for B sequences of T tokens (``packed``: T rows in
    all), D channels and N state values; 0 for most sizes."""
    dims = _SCAN.pack(B, T, D, N, groups, 0, 0, 0, 0, 0, 0, 0, 0, 0)
    return int(_qz._lib().gdr_selective_scan_workspace_bytes(dims, 1 if packed else 0))


def selective_scan_step(x, dt, A, B, C, state, D=None, z=None, dt_bias=None, dt_softplus: bool = False, out=None,
                        out_state=None, stream=None):
    """One new token of every sequence through :func:`selective_scan` (gdr_selective_scan_step): ``x``,
    ``dt``, ``z`` are ``[B, D]``, ``B`` and ``C`` ``[B, N]`` or ``[B, G, N]``.  Updates ``state`` in place unless
    ``out_state`` is given.  Returns y.  ``state`` may be None (zeros; ``out_state`` then receives the new
    state if given)."""
    end = state if out_state is None else out_state
    if stream is None:
        status = (_qz._B or _qz._binding()).selective_scan(x, dt, A, B, C, D, z, dt_bias, dt_softplus, state, None, out, end, False,
                                                           True, None)
        if status is not None:
            if status:
                _fail(status)
            return out
    elif out is None and _elsewhere(stream, x):
        return _on(stream, selective_scan_step, x, dt, A, B, C, state, D, z, dt_bias, dt_softplus, out, out_state)
    return _scan("gdr_selective_scan_step", x, dt, A, B, C, D, z, dt_bias, dt_softplus, state, None, out, end, False, stream,
                 None, *_tokens(x))[0]


def _scan(entry, x, dt, A, B, C, D, z, dt_bias, dt_softplus, h0, cu, out, ht, want_state, stream, workspace, seqs, T, lead):
    shape, dtype = x.shape, x.dtype
    ch = shape[-1]
    xc = _code(x, "x")
    if A.dim() != 2 or A.shape[0] != ch or not 1 <= A.shape[1] <= SCAN_MAX_STATES:
        raise ValueError(f"A must be [{ch}, N] with N in 1 .. {SCAN_MAX_STATES}, got {list(A.shape)}")
    N = A.shape[1]
    _need(A, "A", (ch, N), _F32)
    _need(dt, "dt", shape, (dtype, _F32), dense=False)
    G = B.shape[-2] if B.dim() == len(lead) + 2 else 1
    gshape = (*lead, G, N) if B.dim() == len(lead) + 2 else (*lead, N)
    if G < 1 or ch % G:
        raise ValueError(f"the channels ({ch}) must be a multiple of B's groups, got {list(B.shape)}")
    _need(B, "B", gshape, dtype, dense=False)
    _need(C, "C", gshape, dtype, dense=False)
    if z is not None:
        _need(z, "z", shape, dtype, dense=False)
    for name, t in (("D", D), ("dt_bias", dt_bias)):
        if t is not None:
            _need(t, name, (ch,), _F32)
    if h0 is not None:
        _need(h0, "h0", (seqs, ch, N), _F32)
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=x.device)
    _need(out, "out", shape, dtype, dense=False)
    if ht is None and want_state:
        ht = torch.empty((seqs, ch, N), dtype=_F32, device=x.device)
    if ht is not None:
        _need(ht, "ht", (seqs, ch, N), _F32)
    tail = len(gshape) - len(lead)
    dims = _SCAN.pack(seqs, T, ch, N, G, xc, _code(dt, "dt"), 1 if dt_softplus else 0, _stride(x, "x"), _stride(dt, "dt"),
                      0 if z is None else _stride(z, "z"), _stride(B, "B", tail), _stride(C, "C", tail), _stride(out, "out"))
    step = entry == "gdr_selective_scan_step"
    need = 0 if step else _qz._lib().gdr_selective_scan_workspace_bytes(dims, cu is not None)
    if workspace is None and need:
        workspace = _workspace(need, x, stream)
    if workspace is not None:
        if workspace.dtype is not torch.uint8:
            raise TypeError(f"workspace must be torch.uint8, got {workspace.dtype}")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    s = _stream(stream, x.get_device(), _SCAN_NAMES, (x, dt, A, B, C, D, z, dt_bias, h0, cu, out, ht, workspace))
    ptrs = [_ptr(t) for t in (x, dt, A, B, C, D, z, dt_bias, h0, out, ht)]
    if step:
        status = _qz._lib().gdr_selective_scan_step(dims, *ptrs, s)
    else:
        status = _qz._lib().gdr_selective_scan(dims, _ptr(cu), *ptrs, _ptr(workspace),
                                               0 if workspace is None else workspace.numel(), s)
    if status:
        _fail(status)
    return out, ht


def _workspace(need, x, stream):
    """Memory of the stream that writes it."""
    def make():
        return torch.empty(need, dtype=torch.uint8, device=x.device)
    return make() if stream is None or not _elsewhere(stream, x) else _on(stream, make)


_SCAN_NAMES = ("x", "dt", "A", "B", "C", "D", "z", "dt_bias", "h0", "cu_seqlens", "out", "ht", "workspace")
