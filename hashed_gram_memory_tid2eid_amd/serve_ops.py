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

from . import _check, _lib, _need
from .train_ops import _INT, _WIDE, _flat, _launch_stream, _matrix, _work

_I32, _U8 = torch.int32, torch.uint8


def _serve_stream(stream, *tensors):
    """The raw stream of a call whose tensors must all live on the current device."""
    raw = _launch_stream(stream, *tensors)
    for t in tensors:
        if t is not None:
            if t.get_device() != torch.cuda.current_device():
                raise ValueError(f"tensors on device {t.get_device()}, the current device is {torch.cuda.current_device()}")
            break
    return raw


def _count(n, name):
    """A whole number that a 32-bit argument holds."""
    n = int(n)
    _need(0 <= n < 1 << 31, f"{name} must be in [0, 2^31), got {n}")
    return n


def _of(t, name, dtype, least):
    """Pointer of a contiguous device tensor of at least so many elements, or None."""
    if t is None:
        return None
    p = _flat(t, name, dtype)
    _need(t.numel() >= least, f"{name} too small")
    return p


def _tables(t, name, rows):
    p, n, blocks, ld, _ = _matrix(t, name, _INT)
    _need(n == rows, f"{name} must have {rows} rows")
    return p, blocks, ld


def _pool(free, name, num_pages):
    return _of(free, name, _I32, (num_pages + 31) // 32)


def engram_block_plan(past, new, tables, free, *, page_size, num_pages, cu_seqlens, token_slots, positions=None,
                      seq_start=None, lens=None, free_out=None, stream=None):
    """Block tables and slot maps from request lengths: past, new int32 [R]; tables int32
    [R][blocks] (updated); free the pool (updated, or left as it is with free_out, which
    receives it).  Writes cu_seqlens [R + 1], token_slots int64 [T] and, where given, positions
    int32 [T], seq_start uint8 [R], lens int32 [R] (may be past); T is token_slots' size."""
    R, T = past.numel(), _count(token_slots.numel(), "T")
    page_size, num_pages = _count(page_size, "page_size"), _count(num_pages, "num_pages")
    _need(new.numel() == R, "past and new must be of one size")
    tp, blocks, ld = _tables(tables, "tables", R)
    out = free if free_out is None else free_out
    _check(_lib.engram_block_plan(
        _of(past, "past", _I32, R), _of(new, "new", _I32, R), R, page_size, tp, ld, blocks, _pool(free, "free", num_pages),
        _pool(out, "free_out", num_pages), num_pages, _of(cu_seqlens, "cu_seqlens", _I32, R + 1),
        _of(seq_start, "seq_start", _U8, R), _of(lens, "lens", _I32, R), T, _of(positions, "positions", _I32, T),
        _of(token_slots, "token_slots", torch.int64, T),
        _serve_stream(stream, past, new, tables, free, out, cu_seqlens, seq_start, lens, positions, token_slots)),
        "engram_block_plan")


def engram_block_release(tables, lens, flags, free, *, page_size, num_pages, stream=None):
    """The pages of rows with a flag become free: tables int32 [R][blocks], lens int32 [R],
    flags uint8 [R]; free is updated."""
    R = _count(lens.numel(), "R")
    page_size, num_pages = _count(page_size, "page_size"), _count(num_pages, "num_pages")
    tp, blocks, ld = _tables(tables, "tables", R)
    _check(_lib.engram_block_release(tp, ld, blocks, _of(lens, "lens", _I32, R), _of(flags, "flags", _U8, R), R, page_size,
                                     _pool(free, "free", num_pages), num_pages,
                                     _serve_stream(stream, tables, lens, flags, free)), "engram_block_release")


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
    _need(scores.dim() == 2 and tokens.dim() == 2, "scores must be [G][K], tokens [G][n]")
    (G, K), n = scores.shape, tokens.shape[1]
    lp, rows, V, ld, kind = _matrix(logits, "logits", _WIDE)
    _need(rows == G * K, "logits must have a row for every beam")
    _need(-1 <= end_token < 1 << 31, "end_token must be a token or -1")
    _count(G, "G"), _count(V, "V")
    for t, name in ((tokens, "tokens"), (parents, "parents"), (out_scores, "out_scores"), (done_out, "done_out")):
        _need(t is None or t.shape == (G, n), f"{name} must be [G][n]")
    _need(done is None or done.shape == (G, K), "done must be [G][K]")
    wp, wn = _work(workspace)
    _check(_lib.engram_beam_select(
        lp, kind, ld, G, K, V, _flat(scores, "scores", torch.float32), None if done is None else _flat(done, "done", _U8),
        end_token, n, _flat(tokens, "tokens", _I32), _flat(parents, "parents", _I32),
        _flat(out_scores, "out_scores", torch.float32), None if done_out is None else _flat(done_out, "done_out", _U8), wp, wn,
        _serve_stream(stream, logits, scores, tokens, parents, out_scores, done, done_out, workspace)),
        "engram_beam_select")


def engram_beam_reorder(parents, *, slots=None, slots_out=None, store=None, slot_src=None, slot_dst=None, tables=None,
                        tables_out=None, lens=None, page_size=None, num_pages=None, free=None, page_src=None, page_dst=None,
                        stream=None):
    """States follow parents int32 [G][K]: slots int32 [G][K] (into slots_out, or in place; the
    entries of ``store``, a Store, with them) and block tables int32 [G * K][blocks] with lens
    int32 [G * K] (into tables_out, or in place; pages that nothing names any more come back to
    free).  slot_src / slot_dst and page_src / page_dst int32 [G][K] receive the rows to copy."""
    _need(parents.dim() == 2, "parents must be [G][K]")
    G, K = parents.shape
    n = _count(G * K, "G * K")
    if slots_out is None:
        slots_out = slots
    tp = op = None
    blocks = ld = 0
    if tables is not None:
        tp, blocks, ld = _tables(tables, "tables", n)
        op, out_blocks, out_ld = (tp, blocks, ld) if tables_out is None else _tables(tables_out, "tables_out", n)
        _need(out_blocks == blocks and (out_ld == ld or n <= 1), "tables_out must be laid out as tables")
        _need(lens is not None and page_size is not None and num_pages is not None,
              "tables need lens, page_size and num_pages")
        page_size, num_pages = _count(page_size, "page_size"), _count(num_pages, "num_pages")
    else:
        _need(tables_out is None and free is None and page_src is None and page_dst is None, "pages need tables")
        page_size = num_pages = 0
    _check(_lib.engram_beam_reorder(
        _of(parents, "parents", _I32, n), G, K, None if store is None else store.handle, _of(slots, "slots", _I32, n),
        _of(slots_out, "slots_out", _I32, n), _of(slot_src, "slot_src", _I32, n), _of(slot_dst, "slot_dst", _I32, n), tp, op,
        ld, blocks, _of(lens, "lens", _I32, n), page_size, None if free is None else _pool(free, "free", num_pages),
        num_pages, _of(page_src, "page_src", _I32, n), _of(page_dst, "page_dst", _I32, n),
        _serve_stream(stream, parents, slots, slots_out, slot_src, slot_dst, tables, tables_out, lens, free, page_src,
                      page_dst)), "engram_beam_reorder")


def engram_state_copy(state, src, dst, *, stream=None):
    """Rows src -> dst (int32 [n], -1 for none) of state [rows][width] or, in every plane,
    [planes][rows][width]; any type, the last dimension contiguous."""
    if not isinstance(state, torch.Tensor):
        raise TypeError("state must be a tensor")
    if not state.is_cuda:
        raise TypeError("state must be a device tensor")
    _need(state.dim() in (2, 3), "state must be [rows][width] or [planes][rows][width]")
    rows, width = state.shape[-2:]
    size = state.element_size()
    strides = state.stride()
    _need(width == 0 or strides[-1] == 1 or width == 1, "state must have contiguous rows")
    pitch = width if rows <= 1 else strides[-2]
    _need(pitch >= width, "state must not have overlapping rows")
    planes = state.shape[0] if state.dim() == 3 else 1
    plane = strides[0] if planes > 1 else 0
    _need(planes <= 1 or plane >= (rows - 1) * pitch + width or pitch >= (planes - 1) * plane + width > width,
          "state must not have overlapping planes")
    n = _count(src.numel(), "n")
    _need(dst.numel() == n, "src and dst must be of one size")
    sp, dp = _flat(src, "src", _I32), _flat(dst, "dst", _I32)
    raw = _serve_stream(stream, state, src, dst)
    if width == 0 or n == 0:
        return
    _check(_lib.engram_state_copy(state.data_ptr(), planes, plane * size, rows, pitch * size, width * size, sp, dp, n, raw),
           "engram_state_copy")
