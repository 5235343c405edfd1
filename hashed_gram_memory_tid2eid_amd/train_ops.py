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
    """(pointer, leading dimension) of a device matrix whose rows are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in types:
        raise TypeError(f"{name} must be one of {[str(x) for x in types]}, got {t.dtype}")
    if not t.is_cuda:
        raise TypeError(f"{name} must be a device tensor")
    _need(t.dim() == 2, f"{name} must be a matrix")
    _need(t.shape[1] <= 1 or t.stride(1) == 1, f"{name} must have contiguous rows")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    _need(ld >= t.shape[1], f"{name} must not have overlapping rows")
    return t.data_ptr(), ld


def _same_device(*tensors):
    devices = {t.device for t in tensors if t is not None}
    _need(len(devices) <= 1, f"tensors on different devices: {sorted(map(str, devices))}")


def _work(workspace):
    if workspace is None:
        return None, 0
    return _dev(workspace, None, "workspace"), workspace.numel() * workspace.element_size()


def _ids(ids):
    """(pointer, T, columns, leading dimension) of int32 ids [T] or [T][columns]."""
    m = ids.unsqueeze(1) if isinstance(ids, torch.Tensor) and ids.dim() == 1 else ids
    p, ld = _matrix(m, "ids", (torch.int32,))
    _need(m.shape[1] >= 1, "ids need a column")
    return p, m.shape[0], m.shape[1], ld


def engram_embed(table, ids, out, *, scale=1.0, seg_pitch=None, stream=None):
    """out[t][c * seg_pitch + d] = scale * table[ids[t][c]][d]; ids int32 [T] or [T][columns],
    -1 for none; seg_pitch defaults to the table's width."""
    tp, table_ld = _matrix(table, "table", _WIDE)
    ip, T, cols, ids_ld = _ids(ids)
    op, out_ld = _matrix(out, "out", _WIDE)
    _same_device(table, ids, out)
    seg = table.shape[1] if seg_pitch is None else int(seg_pitch)
    _need(out.shape[0] >= T and out.shape[1] >= cols * seg, "out too small")
    _check(_lib.engram_embed(tp, _WIDE[table.dtype], table.shape[0], table.shape[1], table_ld, ip, T, cols, ids_ld,
                             float(scale), op, _WIDE[out.dtype], out_ld, seg, _stream(stream)), "engram_embed")


def engram_embed_grad_workspace(places: int, rows: int, dim: int) -> int:
    """Bytes of scratch a gradient of ``places`` = T * columns ids needs."""
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
    dp, dout_ld = _matrix(dout, "dout", _WIDE)
    gp, grad_ld = _matrix(grad, "grad", _WIDE)
    _same_device(ids, dout, grad, unique, count, workspace)
    dim = grad.shape[1]
    seg = dim if seg_pitch is None else int(seg_pitch)
    _need(dout.shape[0] >= T and dout.shape[1] >= cols * seg, "dout too small")
    _need(grad.shape[0] >= (T * cols if mode == "sparse" else rows), "grad has too few rows")
    up = cp = None
    if mode == "sparse":
        _need(unique is not None and count is not None, "a sparse gradient needs unique and count")
        _need(unique.numel() >= T * cols and count.numel() >= 1, "unique / count too small")
        up, cp = _dev(unique, torch.int32, "unique"), _dev(count, torch.int32, "count")
    wp, wn = _work(workspace)
    _check(_lib.engram_embed_grad(ip, T, cols, ids_ld, int(rows), dim, float(scale), dp, _WIDE[dout.dtype], dout_ld, seg,
                                  _GRAD_MODES[mode], gp, _WIDE[grad.dtype], grad_ld, up, cp, wp, wn, _stream(stream)),
           "engram_embed_grad")


_CODES = (torch.float8_e4m3fn, torch.uint8)


def _blocks(n):
    return -(-n // 128)


def _codes_and_scales(q, scales, n, k, block, name):
    """(codes pointer, leading dimension, scales pointer, scale kind) of an n x k operand."""
    if q is None:
        _need(scales is None, f"{name} scales without codes")
        return None, 0, None, None
    _need(scales is not None, f"{name} codes need scales")
    p, ld = _matrix(q, name, _CODES)
    _need(q.shape[0] >= n and q.shape[1] >= 128 * _blocks(k), f"{name} codes too small")
    if scales.dtype not in _SCALES:
        raise TypeError(f"{name} scales must be float32, or uint8 (e8m0)")
    want = (_blocks(k), n if block == 1 else _blocks(n))
    _need(tuple(scales.shape) == want, f"{name} scales must be {list(want)}, got {list(scales.shape)}")
    return p, ld, _dev(scales, None, f"{name} scales"), _SCALES[scales.dtype]


def engram_fp8_quantize(x, q, scales, *, q_t=None, scales_t=None, block_rows=1, stream=None):
    """e4m3fn codes and scales of x [M][K]: q [M][K up to 128s] with scales [K/128][M], and / or
    the transpose q_t [K][M up to 128s] with scales_t [M/128][K]; block_rows=128 takes one scale
    per 128 x 128 (scales [K/128][M/128])."""
    _need(block_rows in (1, 128), "block_rows must be 1 or 128")
    xp, x_ld = _matrix(x, "x", _WIDE)
    M, K = x.shape
    _need(q is not None or q_t is not None, "no output: give q or q_t")
    qp, q_ld, sp, kind = _codes_and_scales(q, scales, M, K, block_rows, "q")
    tp, t_ld, stp, kind_t = _codes_and_scales(q_t, scales_t, K, M, block_rows, "q_t")
    _need(kind is None or kind_t is None or kind == kind_t, "both scales must be of one type")
    _same_device(x, q, scales, q_t, scales_t)
    _check(_lib.engram_fp8_quantize(xp, _WIDE[x.dtype], M, K, x_ld, kind if kind is not None else kind_t, block_rows, qp,
                                    q_ld, sp, tp, t_ld, stp, _stream(stream)), "engram_fp8_quantize")


def engram_fp8_matmul_workspace(M: int, N: int, K: int) -> int:
    """Bytes of scratch an M x N product over K (rounded up to whole blocks) needs."""
    n = ctypes.c_int64(0)
    _check(_lib.engram_fp8_matmul_workspace(int(M), int(N), 128 * _blocks(int(K)), ctypes.byref(n)),
           "engram_fp8_matmul_workspace")
    return int(n.value)


def engram_fp8_matmul(a, scales_a, b, scales_b, out, *, workspace=None, stream=None):
    """out[m][n] = sum_k a[m][k] b[n][k] of quantised operands: a [M][K] with scales [K/128][M],
    b [N][K] with scales [K/128][N] or [K/128][N/128]; K whole blocks of 128."""
    op, out_ld = _matrix(out, "out", _WIDE)
    M, N = out.shape
    _need(isinstance(a, torch.Tensor) and isinstance(b, torch.Tensor) and a.dim() == 2 and b.dim() == 2,
          "a and b must be matrices")
    K = a.shape[1]
    _need(K % 128 == 0 and K > 0 and b.shape[1] == K, "a and b need the same K, whole blocks of 128")
    _need(a.shape[0] == M and b.shape[0] == N, "out must be [rows of a][rows of b]")
    block = 1 if scales_b.dim() == 2 and scales_b.shape[1] == N else 128
    ap, a_ld, sap, kind = _codes_and_scales(a, scales_a, M, K, 1, "a")
    bp, b_ld, sbp, kind_b = _codes_and_scales(b, scales_b, N, K, block, "b")
    _need(kind == kind_b, "both scales must be of one type")
    _same_device(a, scales_a, b, scales_b, out, workspace)
    wp, wn = _work(workspace)
    _check(_lib.engram_fp8_matmul(ap, a_ld, sap, bp, b_ld, sbp, block, kind, M, N, K, op, _WIDE[out.dtype], out_ld, wp, wn,
                                  _stream(stream)), "engram_fp8_matmul")


def engram_gate_add_backward(v, streams, dy, dx, dv, *, keep=None, T=None, stream=None):
    """Gradients of engram_gate_add: dx of the streams [T][hc][hidden] before the add (dx may be
    dy) and dv of v, from the streams before the add and dy of the streams after it."""
    if T is None:
        T = streams.shape[0]
    _need(streams.dim() == 3 and streams.shape[0] >= T, "streams must be [T][hc][hidden]")
    hc, hidden = streams.shape[1], streams.shape[2]
    for t, name in ((dy, "dy"), (dx, "dx")):
        _need(t.dim() == 3 and t.shape[0] >= T and t.shape[1:] == streams.shape[1:], f"{name} must be [T][hc][hidden]")
    for t, name in ((v, "v"), (dv, "dv")):
        _need(t.dim() == 2 and t.shape[0] >= T and t.shape[1] == hidden, f"{name} must be [T][hidden]")
    _need(keep is None or keep.numel() >= T, "keep too small")
    _same_device(v, streams, dy, dx, dv, keep)
    _check(_lib.engram_gate_add_backward(
        _dev(v, torch.float32, "v"), _dev(streams, torch.bfloat16, "streams"), _dev(keep, torch.uint8, "keep"),
        _dev(dy, torch.bfloat16, "dy"), hidden, hc, _dev(dx, torch.bfloat16, "dx"), _dev(dv, torch.float32, "dv"), T,
        _stream(stream)), "engram_gate_add_backward")
