"""The operators of ``include/kda_ops.h``: int8 rows (:func:`quant_rows`), the
projections on them (:func:`linear_i8`) and linear attention with a decay a
head, one token at a time (:func:`la_step`) and over prompts
(:func:`la_prefill`).  Like the rest of the package this only marshals
arguments; everything runs in the kernels of ``libkda.so``.

Each takes CUDA tensors of one device, which need not be the current one, and
enqueues on that device's current stream, or on ``stream`` (a raw handle), which
then owns the results that are not given: use them there, or on streams that wait for it.
"""
from __future__ import annotations

import ctypes

import torch

from . import HEAD_DIM, KdaError, _current_stream, load_library

_BF16, _F32, _I8, _I32 = torch.bfloat16, torch.float32, torch.int8, torch.int32
_STATE = {_F32: 0, _BF16: 1}  # KDA_STATE_F32, KDA_STATE_BF16


def _call(name, device, stream, *args):
    """The C function on the tensors' device, on `stream` or its current one."""
    fn = getattr(load_library(), name)
    if stream is None:
        stream = _current_stream(device)
    if device.index == torch._C._cuda_getDevice():
        rc = fn(*args, stream or None)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream or None)
    if rc != 0:
        raise KdaError(name, rc)


def _empty(shape, dtype, device, stream):
    """Memory that a call on `stream` writes: owned by that stream, so that it was not handed on too early."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _check(name, stream, device):
    with torch.cuda.device(device):
        flags = ctypes.c_uint(0)
        rc = getattr(load_library(), name)(stream or torch.cuda.current_stream().cuda_stream or None,
                                           ctypes.byref(flags))
    if rc != 0:
        raise KdaError(name, rc)
    return flags.value


def kda_linear_i8_check(stream: int = 0, device=None) -> int:
    """Synchronise `stream` (0: the current one), return and clear linear_i8's error bits on `device`."""
    return _check("kda_linear_i8_check", stream, device)


def kda_la_check(stream: int = 0, device=None) -> int:
    """Synchronise `stream` (0: the current one), return and clear la_step's and la_prefill's error bits
    (KDA_ERR_SLOT, KDA_ERR_SEQ, KDA_ERR_TIMEOUT) on `device`."""
    return _check("kda_la_check", stream, device)


def _refuse(t, name, dtype, device, shape, layout):
    """What is wrong with an argument that its one-line check has turned down."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    raise ValueError(f"{name} must be {shape} {layout}, got shape {list(t.shape)} with strides {list(t.stride())}")


def _cuda(t, name, dtype):
    """The device of the tensor that the others of a call are compared with."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype:
        _refuse(t, name, dtype, None, "", "")
    return t.device


def _matrix(t, name, dtype, device, shape=None):
    """The row stride of a matrix with unit column stride (a row by itself has none to speak of)."""
    if isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.dim() == 2:
        rows, cols = t.shape
        if shape is None or (rows, cols) == shape:
            ld, unit = t.stride()
            if unit == 1 or cols == 1:
                return ld if rows > 1 else cols
    _refuse(t, name, dtype, device, list(shape) if shape else "[rows, columns]", "with unit column stride")


def _vector(t, name, dtype, device, n):
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.dim() == 1
            and t.shape[0] == n and (n < 2 or t.stride(0) == 1)):
        _refuse(t, name, dtype, device, [n], "and contiguous")


def quant_rows(x, residual=None, norm_weight=None, *, eps: float = 1e-6, out=None, scales=None, stream=None):
    """int8 rows with one fp32 scale each: ``(q, scales)`` with ``q * scales[:, None]``
    the RMSNorm of ``h = x + residual`` (``norm_weight`` given) or ``h`` itself.

    x [rows, cols] bf16 with unit column stride; ``residual`` likewise, replaced
    by h (bf16); ``norm_weight`` [cols] bf16.  cols a multiple of 16 up to 32768.
    ``out`` int8 [rows, cols] and ``scales`` fp32 [rows] are made if not given.
    A row with a NaN or an infinity has scale NaN."""
    device = _cuda(x, "x", _BF16)
    ldx = _matrix(x, "x", _BF16, device)
    rows, cols = shape = tuple(x.shape)
    res = weight = None
    ldr = 0
    if residual is not None:
        ldr = _matrix(residual, "residual", _BF16, device, shape)
        res = residual.data_ptr()
    if norm_weight is not None:
        _vector(norm_weight, "norm_weight", _BF16, device, cols)
        weight = norm_weight.data_ptr()
    if out is None:
        out = _empty(shape, _I8, device, stream)
    ldq = _matrix(out, "out", _I8, device, shape)
    if scales is None:
        scales = _empty((rows,), _F32, device, stream)
    _vector(scales, "scales", _F32, device, rows)
    _call("kda_quant_rows", device, stream, x.data_ptr(), rows, ldx, cols, res, ldr, weight, eps, out.data_ptr(), ldq,
          scales.data_ptr())
    return out, scales


def linear_i8(x, x_scales, w, w_scales, out=None, *, stream=None):
    """y = (x @ w.T) * x_scales[:, None] * w_scales, bf16, for int8 x [rows, K]
    (unit column stride) and w [N, K] (contiguous) and fp32 scales [rows] and
    [N]; K a multiple of 16.  ``out`` [rows, N] bf16 or None."""
    device = _cuda(x, "x", _I8)
    ldx = _matrix(x, "x", _I8, device)
    rows, K = x.shape
    if _matrix(w, "w", _I8, device) != K or w.shape[1] != K:
        raise ValueError("w must be a contiguous [N, K] with x's K")
    N = w.shape[0]
    _vector(x_scales, "x_scales", _F32, device, rows)
    _vector(w_scales, "w_scales", _F32, device, N)
    if out is None:
        out = _empty((rows, N), _BF16, device, stream)
    ldy = _matrix(out, "out", _BF16, device, (rows, N))
    _call("kda_linear_i8", device, stream, x.data_ptr(), rows, ldx, x_scales.data_ptr(), w.data_ptr(),
          w_scales.data_ptr(), N, K, out.data_ptr(), ldy)
    return out


def _heads(t, name, rows, device):
    """(heads, row stride) of [rows, heads, 128] bf16 with the heads of a row side by side."""
    if isinstance(t, torch.Tensor) and t.dtype == _BF16 and t.device == device and t.dim() == 3:
        n, heads, d = t.shape
        ld, head, unit = t.stride()
        if n == rows and d == HEAD_DIM and heads > 0 and unit == 1 and (head == HEAD_DIM or heads == 1):
            return heads, ld if rows > 1 else heads * HEAD_DIM
    _refuse(t, name, _BF16, device, f"[{rows}, heads, {HEAD_DIM}]", "with strides [row, 128, 1]")


def _attention(q, k, v, g, state, slots, scale, out, stream):
    """The arguments that step and prompt share, checked."""
    device = _cuda(v, "v", _BF16)
    rows = v.shape[0]
    heads, ldv = _heads(v, "v", rows, device)
    qk_heads, ldq = _heads(q, "q", rows, device)
    k_heads, ldk = _heads(k, "k", rows, device)
    if k_heads != qk_heads or heads % qk_heads:
        raise ValueError("q and k need the same heads, a divisor of v's")
    ldg = 0
    if isinstance(g, torch.Tensor) and g.dim() == 2:
        ldg = _matrix(g, "g", _F32, device, (rows, heads))
        if 0 < ldg < heads:
            raise ValueError("g: one decay a head for every token is a [heads] vector")
    else:
        _vector(g, "g", _F32, device, heads)
    pool = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() == 4 else 0
    if (not pool or state.dtype not in _STATE or state.device != device or not state.is_contiguous()
            or tuple(state.shape) != (pool, heads, HEAD_DIM, HEAD_DIM)):
        if isinstance(state, torch.Tensor) and state.dtype not in _STATE:
            raise TypeError("state must be a float32 or bfloat16 tensor")
        _refuse(state, "state", state.dtype if isinstance(state, torch.Tensor) else _F32, device,
                f"[pool, {heads}, 128, 128]", "and contiguous")
    if not (isinstance(slots, torch.Tensor) and slots.dtype == _I32 and slots.device == device and slots.dim() == 1
            and slots.is_contiguous()):
        _refuse(slots, "slots", _I32, device, "[slots]", "and contiguous")
    if out is None:
        out = _empty((rows, heads, HEAD_DIM), _BF16, device, stream)
    out_heads, ldo = _heads(out, "out", rows, device)
    if out_heads != heads:
        raise ValueError("out must be v's [rows, heads, 128]")
    args = (q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, rows, heads, qk_heads, g.data_ptr(), ldg,
            HEAD_DIM ** -0.5 if scale is None else scale)
    return device, rows, heads, pool, args, out, ldo


def la_step(q, k, v, g, *, state, slots, scale=None, out=None, stream=None):
    """One token of linear attention with a decay a head for each row:
    ``S = exp(g) S + v k^T; out = scale S q`` on the states ``state[slots]``, updated
    in place.

    q, k [rows, qk_heads, 128] and v [rows, heads, 128] bf16 (views of one packed
    row will do), g fp32 [heads] or [rows, heads] (log decays, <= 0), state
    [pool, heads, 128 (v), 128 (k)] fp32 or bf16, slots int32 [>= rows] (-1: a padding
    row).  ``scale`` is 128 ** -0.5 unless given.  Returns out [rows, heads, 128]."""
    device, rows, _, pool, args, out, ldo = _attention(q, k, v, g, state, slots, scale, out, stream)
    if slots.shape[0] < rows:
        raise ValueError("slots needs an entry for each row")
    _call("kda_la_step", device, stream, *args, state.data_ptr(), _STATE[state.dtype], pool, slots.data_ptr(),
          out.data_ptr(), ldo)
    return out


def la_prefill(q, k, v, g, *, state, slots, cu_seqlens, max_len, has_state=None, scale=None, out=None,
               workspace=None, stream=None):
    """The tokens of packed prompts through the attention of :func:`la_step`:
    sequence i has the rows ``cu_seqlens[i]:cu_seqlens[i + 1]``, starts from
    ``state[slots[i]]`` where ``has_state[i]`` is nonzero and from zeros
    elsewhere, and leaves its last state there.

    ``cu_seqlens`` int32 [seqs + 1] and ``has_state`` int32 [seqs] (None: every
    sequence is new) are read on the GPU; ``max_len`` is a bound on the lengths.
    ``workspace`` (uint8, ``la_prefill_workspace`` bytes) is made if not given.
    The other arguments are as in :func:`la_step`, slots by sequence.  Rows of
    ``out`` behind the last sequence are left as they are."""
    device, rows, heads, pool, args, out, ldo = _attention(q, k, v, g, state, slots, scale, out, stream)
    if not (isinstance(cu_seqlens, torch.Tensor) and cu_seqlens.dtype == _I32 and cu_seqlens.device == device
            and cu_seqlens.dim() == 1 and cu_seqlens.shape[0] > 0 and cu_seqlens.is_contiguous()):
        _refuse(cu_seqlens, "cu_seqlens", _I32, device, "[seqs + 1]", "and contiguous")
    seqs = cu_seqlens.shape[0] - 1
    if slots.shape[0] < seqs:
        raise ValueError("slots needs an entry for each sequence")
    has = None
    if has_state is not None:
        _vector(has_state, "has_state", _I32, device, seqs)
        has = has_state.data_ptr()
    max_len = int(max_len)
    if max_len < 0:
        raise ValueError("max_len must not be negative")
    # (a chunk of 128 tokens is never cut: the shortest calls need not ask)
    need = la_prefill_workspace(rows, heads, seqs, max_len, device=device) if max_len > 128 else 0
    if workspace is not None:
        if not (isinstance(workspace, torch.Tensor) and workspace.dtype == torch.uint8 and workspace.device == device
                and workspace.is_contiguous() and workspace.numel() >= need):
            _refuse(workspace, "workspace", torch.uint8, device, f"[>= {need}]", "and contiguous")
    elif need:
        workspace = _empty(need, torch.uint8, device, stream)
    _call("kda_la_prefill", device, stream, *args, cu_seqlens.data_ptr(), seqs, max_len, has, state.data_ptr(),
          _STATE[state.dtype], pool, slots.data_ptr(), out.data_ptr(), ldo,
          workspace.data_ptr() if workspace is not None else None,
          workspace.numel() if workspace is not None else 0)
    return out


def la_prefill_workspace(rows: int, heads: int, seqs: int, max_len: int, device=None) -> int:
    """Bytes of workspace that la_prefill takes for these sizes on `device`."""
    fn = load_library().kda_la_prefill_workspace
    if device is None or device.index == torch._C._cuda_getDevice():
        return fn(rows, heads, seqs, max_len)
    with torch.cuda.device(device):
        return fn(rows, heads, seqs, max_len)
