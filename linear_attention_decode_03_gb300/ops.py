"""The operators of ``include/kda_ops.h``: int8 rows (:func:`quant_rows`), the
projections on them (:func:`linear_i8`) and linear attention with a decay a
head, one token at a time (:func:`la_step`) and over prompts
(:func:`la_prefill`).  Like the rest of the package this only marshals
arguments; everything runs in the kernels of ``libkda.so``.

Each takes CUDA tensors of one device, which need not be the current one, and
enqueues on that device's current stream, or on ``stream`` (a raw handle).
"""
from __future__ import annotations

import ctypes

import torch

_HEAD_DIM = 128
_HAS_DTYPE = {torch.float32: 0, torch.bfloat16: 1}  # KDA_STATE_F32, KDA_STATE_BF16


def _call(name, device, stream, *args):
    """The C function on the tensors' device, on `stream` or its current one."""
    from . import KdaError, _current_stream, load_library

    fn = getattr(load_library(), name)
    if stream is None:
        stream = _current_stream(device)
    if device.index == torch.cuda.current_device():
        rc = fn(*args, stream or None)
    else:
        with torch.cuda.device(device):
            rc = fn(*args, stream or None)
    if rc != 0:
        raise KdaError(name, rc)


def _check(name, stream, device):
    from . import KdaError, load_library

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


def _want(t, name, dtype, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _matrix(t, name, dtype, device, shape=None):
    """A matrix with unit column stride; its row stride."""
    _want(t, name, dtype, device)
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] > 1) or (shape is not None and tuple(t.shape) != shape):
        raise ValueError(f"{name} must be {list(shape) if shape else '[rows, columns]'} with unit column stride")
    # a row by itself has no stride to speak of
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _vector(t, name, dtype, device, n):
    _want(t, name, dtype, device)
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}]")


def quant_rows(x, residual=None, norm_weight=None, *, eps: float = 1e-6, out=None, scales=None, stream=None):
    """int8 rows with one fp32 scale each: ``(q, scales)`` with ``q * scales[:, None]``
    the RMSNorm of ``h = x + residual`` (``norm_weight`` given) or ``h`` itself.

    x [rows, cols] bf16 with unit column stride; ``residual`` likewise, replaced
    by h (bf16); ``norm_weight`` [cols] bf16.  cols a multiple of 16 up to 32768.
    ``out`` int8 [rows, cols] and ``scales`` fp32 [rows] are made if not given.
    A row with a NaN or an infinity has scale NaN."""
    _want(x, "x", torch.bfloat16)
    device = x.device
    ldx = _matrix(x, "x", torch.bfloat16, device)
    rows, cols = x.shape
    ldr = 0
    if residual is not None:
        ldr = _matrix(residual, "residual", torch.bfloat16, device, (rows, cols))
    if norm_weight is not None:
        _vector(norm_weight, "norm_weight", torch.bfloat16, device, cols)
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.int8, device=device)
    ldq = _matrix(out, "out", torch.int8, device, (rows, cols))
    if scales is None:
        scales = torch.empty((rows,), dtype=torch.float32, device=device)
    _vector(scales, "scales", torch.float32, device, rows)
    _call("kda_quant_rows", device, stream, x.data_ptr(), rows, ldx, cols,
          residual.data_ptr() if residual is not None else None, ldr,
          norm_weight.data_ptr() if norm_weight is not None else None, eps, out.data_ptr(), ldq, scales.data_ptr())
    return out, scales


def linear_i8(x, x_scales, w, w_scales, out=None, *, stream=None):
    """y = (x @ w.T) * x_scales[:, None] * w_scales, bf16, for int8 x [rows, K]
    (unit column stride) and w [N, K] (contiguous) and fp32 scales [rows] and
    [N]; K a multiple of 16.  ``out`` [rows, N] bf16 or None."""
    _want(x, "x", torch.int8)
    device = x.device
    ldx = _matrix(x, "x", torch.int8, device)
    _want(w, "w", torch.int8, device)
    rows, K = x.shape
    if w.dim() != 2 or not w.is_contiguous() or w.shape[1] != K:
        raise ValueError("w must be a contiguous [N, K] with x's K")
    N = w.shape[0]
    _vector(x_scales, "x_scales", torch.float32, device, rows)
    _vector(w_scales, "w_scales", torch.float32, device, N)
    if out is None:
        out = torch.empty((rows, N), dtype=torch.bfloat16, device=device)
    ldy = _matrix(out, "out", torch.bfloat16, device, (rows, N))
    _call("kda_linear_i8", device, stream, x.data_ptr(), rows, ldx, x_scales.data_ptr(), w.data_ptr(),
          w_scales.data_ptr(), N, K, out.data_ptr(), ldy)
    return out


def _heads(t, name, rows, device):
    """[rows, heads, 128] bf16 with its heads side by side; (heads, row stride)."""
    _want(t, name, torch.bfloat16, device)
    if t.dim() != 3 or t.shape[0] != rows or t.shape[2] != _HEAD_DIM:
        raise ValueError(f"{name} must be [rows, heads, 128]")
    heads = t.shape[1]
    if heads < 1 or t.stride(2) != 1 or (heads > 1 and t.stride(1) != _HEAD_DIM):
        raise ValueError(f"{name} needs its heads' 128 values side by side (strides [row, 128, 1])")
    return heads, t.stride(0) if rows > 1 else heads * _HEAD_DIM


def _attention(q, k, v, g, state, slots, scale, out):
    """The arguments that step and prompt share, checked."""
    _want(v, "v", torch.bfloat16)
    device = v.device
    if v.dim() != 3:
        raise ValueError("v must be [rows, heads, 128]")
    rows = v.shape[0]
    heads, ldv = _heads(v, "v", rows, device)
    qk_heads, ldq = _heads(q, "q", rows, device)
    k_heads, ldk = _heads(k, "k", rows, device)
    if k_heads != qk_heads or heads % qk_heads:
        raise ValueError("q and k need the same heads, a divisor of v's")
    _want(g, "g", torch.float32, device)
    if g.dim() == 1:
        _vector(g, "g", torch.float32, device, heads)
        ldg = 0
    else:
        ldg = _matrix(g, "g", torch.float32, device, (rows, heads))
        if 0 < ldg < heads:
            raise ValueError("g: one decay a head for every token is a [heads] vector")
    if not isinstance(state, torch.Tensor) or state.dtype not in _HAS_DTYPE:
        raise TypeError("state must be a float32 or bfloat16 tensor")
    _want(state, "state", state.dtype, device)
    if state.dim() != 4 or tuple(state.shape[1:]) != (heads, _HEAD_DIM, _HEAD_DIM) or not state.is_contiguous():
        raise ValueError("state must be a contiguous [pool, heads, 128, 128]")
    _want(slots, "slots", torch.int32, device)
    if slots.dim() != 1 or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous vector")
    if out is None:
        out = torch.empty((rows, heads, _HEAD_DIM), dtype=torch.bfloat16, device=device)
    out_heads, ldo = _heads(out, "out", rows, device)
    if out_heads != heads:
        raise ValueError("out must be v's [rows, heads, 128]")
    if scale is None:
        scale = _HEAD_DIM ** -0.5
    args = (q.data_ptr(), ldq, k.data_ptr(), ldk, v.data_ptr(), ldv, rows, heads, qk_heads, g.data_ptr(), ldg, scale)
    return device, rows, heads, args, out, ldo


def la_step(q, k, v, g, *, state, slots, scale=None, out=None, stream=None):
    """One token of linear attention with a decay a head for each row:
    ``S = exp(g) S + v k^T; out = scale S q`` on the states ``state[slots]``, updated
    in place.

    q, k [rows, qk_heads, 128] and v [rows, heads, 128] bf16 (views of one packed
    row will do), g fp32 [heads] or [rows, heads] (log decays, <= 0), state
    [pool, heads, 128 (v), 128 (k)] fp32 or bf16, slots int32 [>= rows] (-1: a padding
    row).  ``scale`` is 128 ** -0.5 unless given.  Returns out [rows, heads, 128]."""
    device, rows, _, args, out, ldo = _attention(q, k, v, g, state, slots, scale, out)
    if slots.shape[0] < rows:
        raise ValueError("slots needs an entry for each row")
    _call("kda_la_step", device, stream, *args, state.data_ptr(), _HAS_DTYPE[state.dtype], state.shape[0],
          slots.data_ptr(), out.data_ptr(), ldo)
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
    device, rows, heads, args, out, ldo = _attention(q, k, v, g, state, slots, scale, out)
    _want(cu_seqlens, "cu_seqlens", torch.int32, device)
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous [seqs + 1]")
    seqs = cu_seqlens.shape[0] - 1
    if slots.shape[0] < seqs:
        raise ValueError("slots needs an entry for each sequence")
    if has_state is not None:
        _vector(has_state, "has_state", torch.int32, device, seqs)
    max_len = int(max_len)
    if max_len < 0:
        raise ValueError("max_len must not be negative")
    need = la_prefill_workspace(rows, heads, seqs, max_len, device=device)
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8, device)
        if not workspace.is_contiguous() or workspace.numel() < need:
            raise ValueError(f"workspace must be contiguous with {need} bytes")
    elif need:
        if stream is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        else:  # owned by the stream that uses it, so that its memory is not handed on too early
            with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device)):
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
    _call("kda_la_prefill", device, stream, *args, cu_seqlens.data_ptr(), seqs, max_len,
          has_state.data_ptr() if has_state is not None else None, state.data_ptr(), _HAS_DTYPE[state.dtype],
          state.shape[0], slots.data_ptr(), out.data_ptr(), ldo,
          workspace.data_ptr() if workspace is not None else None,
          workspace.numel() if workspace is not None else 0)
    return out


def la_prefill_workspace(rows: int, heads: int, seqs: int, max_len: int, device=None) -> int:
    """Bytes of workspace that la_prefill takes for these sizes on `device`."""
    from . import load_library

    lib = load_library()
    if device is None or device.index == torch.cuda.current_device():
        return lib.kda_la_prefill_workspace(rows, heads, seqs, max_len)
    with torch.cuda.device(device):
        return lib.kda_la_prefill_workspace(rows, heads, seqs, max_len)
