"""The serving operators of include/engram.h: marshalling and size checks only.

Lengths, tables, slots and pairs are int32 tensors, flags uint8, a pool of pages an int32
tensor of ceil(num_pages / 32) words whose set bits are free pages.  Block tables may be
row-strided views (their last dimension contiguous); other tensors are contiguous.  Scratch
comes from the caller (``*_workspace`` gives its size in bytes), so that a call allocates
nothing.
"""
from __future__ import annotations

import ctypes

import torch

from . import ENGRAM_DTYPE_BF16, ENGRAM_DTYPE_F32, _check, _lib, _need, _stream

try:
    from ._tensor_args import address as _arg, device as _place, matrix as _rows, torch_version as _torch
    if _torch != torch.__version__:  # it inlines that torch's object layouts
        raise ImportError(f"it was built for torch {_torch}, this is {torch.__version__}")
except ImportError as e:
    _absent = e

    def _place(t, name):
        """The first check of every operator here: without the module none of them can run."""
        raise ImportError("the extension module _tensor_args is missing or does not fit this torch: build it with "
                          "`python hashed_gram_memory_tid2eid_amd/build_lib.py`") from _absent


_I32, _I64, _U8, _F32 = torch.int32, torch.int64, torch.uint8, torch.float32
_LOGITS = {torch.bfloat16: ENGRAM_DTYPE_BF16, torch.float32: ENGRAM_DTYPE_F32}
# (looked up once: 0.1 us a call; a torch without it may still be imported)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _raw(stream, dev):
    return _raw_stream(dev) if stream is None else _stream(stream)


def _count(n, name):
    """A whole number that a 32-bit argument holds."""
    if not 0 <= n < 1 << 31 or n != int(n):
        raise ValueError(f"{name} must be a whole number in [0, 2^31), got {n}")
    return int(n)


def _tables(t, name, rows, dev):
    """(pointer, columns, leading dimension) of a table of so many rows."""
    p, n, blocks, ld = _rows(t, name, _I32, dev)
    if n != rows:
        raise ValueError(f"{name} must have {rows} rows, got {n}")
    return p, blocks, ld


def engram_block_plan(past, new, tables, free, *, page_size, num_pages, cu_seqlens, token_slots, positions=None,
                      seq_start=None, lens=None, free_out=None, stream=None):
    """Block tables and slot maps from request lengths: past, new int32 [R]; tables int32
    [R][blocks] (updated); free the pool (updated, or left as it is with free_out, which
    receives it).  Writes cu_seqlens [R + 1], token_slots int64 [T] and, where given, positions
    int32 [T], seq_start uint8 [R], lens int32 [R] (may be past); T is token_slots' size."""
    dev = _place(past, "past")
    R, T = past.numel(), _count(token_slots.numel(), "T")
    page_size, num_pages = _count(page_size, "page_size"), _count(num_pages, "num_pages")
    words = (num_pages + 31) // 32
    _need(new.numel() == R, "past and new must be of one size")
    tp, blocks, ld = _tables(tables, "tables", R, dev)
    fp = _arg(free, "free", _I32, words, dev)
    _check(_lib.engram_block_plan(
        _arg(past, "past", _I32, R, dev), _arg(new, "new", _I32, R, dev), R, page_size, tp, ld, blocks, fp,
        fp if free_out is None else _arg(free_out, "free_out", _I32, words, dev), num_pages,
        _arg(cu_seqlens, "cu_seqlens", _I32, R + 1, dev), _arg(seq_start, "seq_start", _U8, R, dev),
        _arg(lens, "lens", _I32, R, dev), T, _arg(positions, "positions", _I32, T, dev),
        _arg(token_slots, "token_slots", _I64, T, dev), _raw(stream, dev)), "engram_block_plan")


def engram_block_release(tables, lens, flags, free, *, page_size, num_pages, stream=None):
    """The pages of rows with a flag become free: tables int32 [R][blocks], lens int32 [R],
    flags uint8 [R]; free is updated."""
    dev = _place(lens, "lens")
    R = _count(lens.numel(), "R")
    page_size, num_pages = _count(page_size, "page_size"), _count(num_pages, "num_pages")
    tp, blocks, ld = _tables(tables, "tables", R, dev)
    _check(_lib.engram_block_release(
        tp, ld, blocks, _arg(lens, "lens", _I32, R, dev), _arg(flags, "flags", _U8, R, dev), R, page_size,
        _arg(free, "free", _I32, (num_pages + 31) // 32, dev), num_pages, _raw(stream, dev)), "engram_block_release")


def engram_beam_select_workspace(G: int, K: int, V: int, n: int) -> int:
    """Bytes of scratch that selections of n among V tokens need, for up to ``G`` requests of K beams."""
    size = ctypes.c_int64(0)
    _check(_lib.engram_beam_select_workspace(_count(G, "G"), _count(K, "K"), _count(V, "V"), _count(n, "n"), ctypes.byref(size)),
           "engram_beam_select_workspace")
    return int(size.value)


def engram_beam_select(logits, scores, tokens, parents, out_scores, *, workspace, done=None, done_out=None, end_token=-1,
                       stream=None):
    """The n best continuations of every request's beams: logits [G * K][V] (bf16 or float32,
    rows may be strided), scores float32 [G][K]; tokens, parents int32 [G][n] and out_scores
    float32 [G][n] are written, done_out uint8 [G][n] where given.  done uint8 [G][K] marks
    beams that have ended (end_token is then needed)."""
    dev = _place(scores, "scores")
    _need(scores.dim() == 2 and tokens.dim() == 2, "scores must be [G][K], tokens [G][n]")
    (G, K), shape = scores.shape, tokens.shape
    n = _count(shape[1], "n")
    lp, rows, V, ld = _rows(logits, "logits", None, dev)
    kind = _LOGITS.get(logits.dtype)
    if kind is None:
        raise TypeError(f"logits must be bfloat16 or float32, got {logits.dtype}")
    _need(rows == G * K, "logits must have a row for every beam")
    if shape[0] != G or parents.shape != shape or out_scores.shape != shape:
        raise ValueError("tokens, parents and out_scores must be [G][n]")
    _need(done_out is None or done_out.shape == shape, "done_out must be [G][n]")
    _need(done is None or done.shape == scores.shape, "done must be [G][K]")
    end_token = int(end_token)
    _need(-1 <= end_token < 1 << 31, "end_token must be a token or -1")
    _check(_lib.engram_beam_select(
        lp, kind, ld, G, K, V, _arg(scores, "scores", _F32, 0, dev), _arg(done, "done", _U8, 0, dev), end_token, n,
        _arg(tokens, "tokens", _I32, 0, dev), _arg(parents, "parents", _I32, 0, dev),
        _arg(out_scores, "out_scores", _F32, 0, dev), _arg(done_out, "done_out", _U8, 0, dev),
        _arg(workspace, "workspace", workspace.dtype, 0, dev), workspace.numel() * workspace.element_size(),
        _raw(stream, dev)), "engram_beam_select")


def engram_beam_reorder(parents, *, slots=None, slots_out=None, store=None, slot_src=None, slot_dst=None, tables=None,
                        tables_out=None, lens=None, page_size=None, num_pages=None, free=None, page_src=None, page_dst=None,
                        stream=None):
    """States follow parents int32 [G][K]: slots int32 [G][K] (into slots_out, or in place; the
    entries of ``store``, a Store, with them) and block tables int32 [G * K][blocks] with lens
    int32 [G * K] (into tables_out, or in place; pages that nothing names any more come back to
    free).  slot_src / slot_dst and page_src / page_dst int32 [G][K] receive the rows to copy."""
    dev = _place(parents, "parents")
    _need(parents.dim() == 2, "parents must be [G][K]")
    G, K = parents.shape
    n = _count(G * K, "G * K")
    tp = op = fp = None
    blocks = ld = 0
    if tables is not None:
        tp, blocks, ld = _tables(tables, "tables", n, dev)
        op, out_blocks, out_ld = (tp, blocks, ld) if tables_out is None else _tables(tables_out, "tables_out", n, dev)
        _need(out_blocks == blocks and (out_ld == ld or n <= 1), "tables_out must be laid out as tables")
        _need(lens is not None and page_size is not None and num_pages is not None,
              "tables need lens, page_size and num_pages")
        page_size, num_pages = _count(page_size, "page_size"), _count(num_pages, "num_pages")
        fp = _arg(free, "free", _I32, (num_pages + 31) // 32, dev)
    else:
        _need(tables_out is None and free is None and page_src is None and page_dst is None, "pages need tables")
        page_size = num_pages = 0
    sp = _arg(slots, "slots", _I32, n, dev)
    _check(_lib.engram_beam_reorder(
        _arg(parents, "parents", _I32, n, dev), G, K, None if store is None else store.handle, sp,
        sp if slots_out is None else _arg(slots_out, "slots_out", _I32, n, dev), _arg(slot_src, "slot_src", _I32, n, dev),
        _arg(slot_dst, "slot_dst", _I32, n, dev), tp, op, ld, blocks, _arg(lens, "lens", _I32, n, dev), page_size, fp,
        num_pages, _arg(page_src, "page_src", _I32, n, dev), _arg(page_dst, "page_dst", _I32, n, dev), _raw(stream, dev)),
        "engram_beam_reorder")


def engram_state_copy(state, src, dst, *, stream=None):
    """Rows src -> dst (int32 [n], -1 for none) of state [rows][width] or, in every plane,
    [planes][rows][width]; any type, the last dimension contiguous."""
    dev = _place(state, "state")
    shape, strides, size = state.shape, state.stride(), state.element_size()
    _need(2 <= len(shape) <= 3, "state must be [rows][width] or [planes][rows][width]")
    rows, width = shape[-2], shape[-1]
    _need(width <= 1 or strides[-1] == 1, "state must have contiguous rows")
    pitch = width if rows <= 1 else strides[-2]
    _need(pitch >= width, "state must not have overlapping rows")
    planes, plane = 1, 0
    if len(shape) == 3 and shape[0] != 1:
        planes, plane = shape[0], strides[0]
        _need(planes == 0 or plane >= (rows - 1) * pitch + width or (plane >= width and pitch >= (planes - 1) * plane + width),
              "state must not have overlapping planes")
    n = _count(src.numel(), "n")
    _need(dst.numel() == n, "src and dst must be of one size")
    sp, dp = _arg(src, "src", _I32, n, dev), _arg(dst, "dst", _I32, n, dev)
    if width == 0 or n == 0:
        return
    _check(_lib.engram_state_copy(state.data_ptr(), planes, plane * size, rows, pitch * size, width * size, sp, dp, n,
                                  _raw(stream, dev)), "engram_state_copy")
