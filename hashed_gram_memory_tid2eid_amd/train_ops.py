"""The training operators of include/engram.h: marshalling and size checks only.

Tensors carry the types: a table, an output or a gradient is bfloat16 or float32; codes are
float8_e4m3fn (or uint8) with float32 scales, or uint8 scales for e8m0.  Matrices may be
row-strided views (their last dimension contiguous).  Scratch comes from the caller
(``*_workspace`` gives its size in bytes), so that a call allocates nothing.
"""
from __future__ import annotations

import ctypes

import torch

from . import ENGRAM_DTYPE_BF16, ENGRAM_DTYPE_F32, _check, _dev, _lib, _need, _stream

ENGRAM_GRAD_DENSE, ENGRAM_GRAD_ACCUMULATE, ENGRAM_GRAD_SPARSE = 0, 1, 2
ENGRAM_FP8_SCALE_F32, ENGRAM_FP8_SCALE_E8M0 = 0, 1
_GRAD_MODES = {"dense": ENGRAM_GRAD_DENSE, "accumulate": ENGRAM_GRAD_ACCUMULATE, "sparse": ENGRAM_GRAD_SPARSE}
_WIDE = {torch.bfloat16: ENGRAM_DTYPE_BF16, torch.float32: ENGRAM_DTYPE_F32}
_SCALES = {torch.float32: ENGRAM_FP8_SCALE_F32, torch.uint8: ENGRAM_FP8_SCALE_E8M0}


def _matrix(t, name, types):
    """(pointer, rows, columns, leading dimension, type) of a device matrix whose rows are contiguous."""
    try:
        kind = types[t.dtype]
        rows, cols = t.shape
        ld, step = t.stride()
    except (AttributeError, KeyError, ValueError):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor") from None
        if t.dtype not in types:
            raise TypeError(f"{name} must be one of {[str(x) for x in types]}, got {t.dtype}") from None
        raise ValueError(f"{name} must be a matrix") from None
    if not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"{name} must not have overlapping rows")
    return t.data_ptr(), rows, cols, ld, kind


def _flat(t, name, dtype):
    """Pointer of a contiguous device tensor of one type."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        return _dev(t, dtype, name)  # says what is wrong
    return t.data_ptr()


def _launch_stream(stream, *tensors):
    """The raw stream of a call whose tensors must all live on one device."""
    dev = -1
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev and dev != -1:
                raise ValueError(f"tensors on different devices: {dev} and {d}")
            dev = d
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _work(workspace):
    if workspace is None:
        return None, 0
    return _flat(workspace, "workspace", workspace.dtype), workspace.numel() * workspace.element_size()


_INT = {torch.int32: None}


def _ids(ids):
    """(pointer, T, columns, leading dimension) of int32 ids [T] or [T][columns]."""
    m = ids.unsqueeze(1) if isinstance(ids, torch.Tensor) and ids.dim() == 1 else ids
    p, T, cols, ld, _ = _matrix(m, "ids", _INT)
    _need(cols >= 1, "ids need a column")
    return p, T, cols, ld


def engram_embed(table, ids, out, *, scale=1.0, seg_pitch=None, stream=None):
    """out[t][c * seg_pitch + d] = scale * table[ids[t][c]][d]; ids int32 [T] or [T][columns],
    -1 for none; seg_pitch defaults to the table's width."""
    tp, rows, dim, table_ld, table_type = _matrix(table, "table", _WIDE)
    ip, T, cols, ids_ld = _ids(ids)
    op, out_rows, out_cols, out_ld, out_type = _matrix(out, "out", _WIDE)
    seg = dim if seg_pitch is None else seg_pitch
    _need(out_rows >= T and out_cols >= cols * seg, "out too small")
    _check(_lib.engram_embed(tp, table_type, rows, dim, table_ld, ip, T, cols, ids_ld, scale, op, out_type, out_ld, seg,
                             _launch_stream(stream, table, ids, out)), "engram_embed")


def engram_embed_grad_workspace(places: int, rows: int, dim: int) -> int:
    """Bytes of scratch that gradients of up to ``places`` = T * columns ids need."""
    n = ctypes.c_int64(0)
    _check(_lib.engram_embed_grad_workspace(int(places), int(rows), int(dim), ctypes.byref(n)),
           "engram_embed_grad_workspace")
    return int(n.value)


def engram_embed_grad(ids, dout, grad, *, rows, scale=1.0, mode="dense", seg_pitch=None, unique=None, count=None,
                      workspace=None, stream=None):
    """The gradient of engram_embed for a table of ``rows`` rows, by mode: "dense" writes every
    row of grad [rows][dim], "accumulate" adds to the rows looked up, "sparse" writes one row
    per distinct id into grad [T * columns][dim], the ids into ``unique`` (then -1) and their
    number into ``count``."""
    _need(mode in _GRAD_MODES, f"unknown mode {mode!r}")
    ip, T, cols, ids_ld = _ids(ids)
    dp, dout_rows, dout_cols, dout_ld, dout_type = _matrix(dout, "dout", _WIDE)
    gp, grad_rows, dim, grad_ld, grad_type = _matrix(grad, "grad", _WIDE)
    seg = dim if seg_pitch is None else seg_pitch
    _need(dout_rows >= T and dout_cols >= cols * seg, "dout too small")
    _need(grad_rows >= (T * cols if mode == "sparse" else rows), "grad has too few rows")
    up = cp = None
    if mode == "sparse":
        _need(unique is not None and count is not None, "a sparse gradient needs unique and count")
        up, cp = _flat(unique, "unique", torch.int32), _flat(count, "count", torch.int32)
        _need(unique.numel() >= T * cols and count.numel() >= 1, "unique / count too small")
    wp, wn = _work(workspace)
    _check(_lib.engram_embed_grad(ip, T, cols, ids_ld, rows, dim, scale, dp, dout_type, dout_ld, seg, _GRAD_MODES[mode],
                                  gp, grad_type, grad_ld, up, cp, wp, wn,
                                  _launch_stream(stream, ids, dout, grad, unique, count, workspace)),
           "engram_embed_grad")


_CODES = {torch.float8_e4m3fn: None, torch.uint8: None}


def _blocks(n):
    return -(-n // 128)


def _codes_and_scales(q, scales, n, k, block, name):
    """(codes pointer, leading dimension, scales pointer, scale kind) of an n x k operand."""
    if q is None:
        _need(scales is None, f"{name} scales without codes")
        return None, 0, None, None
    _need(scales is not None, f"{name} codes need scales")
    p, rows, cols, ld, _ = _matrix(q, name, _CODES)
    kb = _blocks(k)
    _need(rows >= n and cols >= 128 * kb, f"{name} codes too small")
    kind = _SCALES.get(scales.dtype)
    if kind is None:
        raise TypeError(f"{name} scales must be float32, or uint8 (e8m0)")
    if scales.shape != (kb, n if block == 1 else _blocks(n)):
        raise ValueError(f"{name} scales must be {[kb, n if block == 1 else _blocks(n)]}, got {list(scales.shape)}")
    return p, ld, _flat(scales, f"{name} scales", scales.dtype), kind


def engram_fp8_quantize(x, q, scales, *, q_t=None, scales_t=None, block_rows=1, stream=None):
    """e4m3fn codes and scales of x [M][K]: q [M][K up to 128s] with scales [K/128][M], and / or
    the transpose q_t [K][M up to 128s] with scales_t [M/128][K]; block_rows=128 takes one scale
    per 128 x 128 (scales [K/128][M/128])."""
    _need(block_rows in (1, 128), "block_rows must be 1 or 128")
    xp, M, K, x_ld, x_type = _matrix(x, "x", _WIDE)
    _need(q is not None or q_t is not None, "no output: give q or q_t")
    qp, q_ld, sp, kind = _codes_and_scales(q, scales, M, K, block_rows, "q")
    tp, t_ld, stp, kind_t = _codes_and_scales(q_t, scales_t, K, M, block_rows, "q_t")
    _need(kind is None or kind_t is None or kind == kind_t, "both scales must be of one type")
    _check(_lib.engram_fp8_quantize(xp, x_type, M, K, x_ld, kind if kind is not None else kind_t, block_rows, qp, q_ld, sp,
                                    tp, t_ld, stp, _launch_stream(stream, x, q, scales, q_t, scales_t)),
           "engram_fp8_quantize")


def engram_fp8_matmul_workspace(M: int, N: int, K: int) -> int:
    """Bytes of scratch an M x N product over K (rounded up to whole blocks) needs."""
    n = ctypes.c_int64(0)
    _check(_lib.engram_fp8_matmul_workspace(int(M), int(N), 128 * _blocks(int(K)), ctypes.byref(n)),
           "engram_fp8_matmul_workspace")
    return int(n.value)


def engram_fp8_matmul(a, scales_a, b, scales_b, out, *, workspace=None, stream=None):
    """out[m][n] = sum_k a[m][k] b[n][k] of quantised operands: a [M][K] with scales [K/128][M],
    b [N][K] with scales [K/128][N] or [K/128][N/128]; K whole blocks of 128."""
    op, M, N, out_ld, out_type = _matrix(out, "out", _WIDE)
    _need(isinstance(a, torch.Tensor) and isinstance(b, torch.Tensor) and a.dim() == 2 and b.dim() == 2,
          "a and b must be matrices")
    (rows_a, K), (rows_b, kb) = a.shape, b.shape
    _need(K % 128 == 0 and K > 0 and kb == K, "a and b need the same K, whole blocks of 128")
    _need(rows_a == M and rows_b == N, "out must be [rows of a][rows of b]")
    block = 1 if scales_b.dim() == 2 and scales_b.shape[1] == N else 128
    ap, a_ld, sap, kind = _codes_and_scales(a, scales_a, M, K, 1, "a")
    bp, b_ld, sbp, kind_b = _codes_and_scales(b, scales_b, N, K, block, "b")
    _need(kind == kind_b, "both scales must be of one type")
    wp, wn = _work(workspace)
    _check(_lib.engram_fp8_matmul(ap, a_ld, sap, bp, b_ld, sbp, block, kind, M, N, K, op, out_type, out_ld, wp, wn,
                                  _launch_stream(stream, a, scales_a, b, scales_b, out, workspace)), "engram_fp8_matmul")


def engram_gate_add_backward(v, streams, dy, dx, dv, *, keep=None, T=None, stream=None):
    """Gradients of engram_gate_add: dx of the streams [T][hc][hidden] before the add (dx may be
    dy) and dv of v, from the streams before the add and dy of the streams after it."""
    _need(streams.dim() == 3, "streams must be [T][hc][hidden]")
    n, hc, hidden = streams.shape
    if T is None:
        T = n
    _need(n >= T, "streams must be [T][hc][hidden]")
    for t, name in ((dy, "dy"), (dx, "dx")):
        shape = t.shape
        _need(len(shape) == 3 and shape[0] >= T and shape[1] == hc and shape[2] == hidden, f"{name} must be [T][hc][hidden]")
    for t, name in ((v, "v"), (dv, "dv")):
        shape = t.shape
        _need(len(shape) == 2 and shape[0] >= T and shape[1] == hidden, f"{name} must be [T][hidden]")
    _need(keep is None or keep.numel() >= T, "keep too small")
    _check(_lib.engram_gate_add_backward(
        _flat(v, "v", torch.float32), _flat(streams, "streams", torch.bfloat16),
        None if keep is None else _flat(keep, "keep", torch.uint8), _flat(dy, "dy", torch.bfloat16), hidden, hc,
        _flat(dx, "dx", torch.bfloat16), _flat(dv, "dv", torch.float32), T,
        _launch_stream(stream, v, streams, dy, dx, dv, keep)), "engram_gate_add_backward")
