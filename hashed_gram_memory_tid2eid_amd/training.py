"""One training step of an Engram site: lookup, 8-bit projection, gate, and all their
gradients, over preallocated device buffers.

``SiteTraining.forward`` looks the call's rows up in trainable tables, quantises them in
blocks of 128 (once along the row for this projection, once transposed for the weight's
gradient), projects them with the 8-bit weight and adds the gated result into the
residual streams.  ``SiteTraining.backward`` takes the gradient of the streams after the
add and leaves the gradient of the streams before it in its place, the weight's gradient
in ``d_weight`` and the tables' in ``table_grads``.  The tables and the float weight are the
caller's; an optimizer steps them and ``load_weight`` takes the new weight over.  ``d_weight`` is
the gradient of the last backward alone, in both modes of the tables' gradients: a caller who
adds up several calls adds it to a sum of its own.

What lies between the operators is kept in few bits where it meets fewer right after.  The
rows are bf16 (of fp32 tables, too): they are only read as e4m3 codes, whose step is 16 times
a bf16 one.  The gradient of the rows is bf16, half its bytes to write and read; it comes from
8-bit operands, each off by up to 2^-4, and the lookup's gradient adds it in fp32.

Every call only enqueues kernels on one stream; nothing is allocated after construction.
"""
from __future__ import annotations

import torch

from . import ENGRAM_TABLE_PER_SITE, Layout, engram_gate_add
from .train_ops import (_flat, engram_embed, engram_embed_grad, engram_embed_grad_workspace, engram_fp8_matmul,
                        engram_fp8_matmul_workspace, engram_fp8_quantize, engram_gate_add_backward)


class SiteTraining:
    """Buffers of one site for calls of up to ``max_tokens`` tokens.

    tables: the site's trainable tables, bf16 or fp32 [rows][D]: one, or one per n-gram
    order, as the layout says.  weight: [hidden][k_pad] bf16 or fp32 (columns of segment
    padding zero).  scales: "f32" or "e8m0".  grad_mode: "sparse" (one row per distinct id;
    the tables may then be of any size) or "accumulate" (added into ``table_grads``, tensors
    like the tables, which the caller clears).  stream: takes the weight over, behind all that
    the current stream holds."""

    def __init__(self, layout: Layout, tables, weight, *, max_tokens: int, embed_scale: float = 1.0,
                 scales: str = "f32", grad_mode: str = "sparse", grad_dtype=torch.float32, hc_mult: int = 4,
                 stream=None):
        info = layout.info
        per_site = info.table_split == ENGRAM_TABLE_PER_SITE
        if len(tables) != (1 if per_site else 3):
            raise ValueError(f"the layout has {1 if per_site else 3} table(s) per site, got {len(tables)}")
        if any(t.dim() != 2 or t.shape[1] != info.row_dim for t in tables):
            raise ValueError(f"tables must be [rows][{info.row_dim}]")
        if any(t.shape[0] < info.rows[n] for n, t in enumerate(tables)):
            raise ValueError("a table has fewer rows than the layout")
        if weight.dim() != 2 or weight.shape[1] != info.k_pad:
            raise ValueError(f"weight must be [hidden][{info.k_pad}] (pad_weight)")
        if scales not in ("f32", "e8m0"):
            raise ValueError(f"unknown scales {scales!r}")
        if grad_mode not in ("sparse", "accumulate"):
            raise ValueError(f"unknown grad_mode {grad_mode!r}")
        if max_tokens < 1:
            raise ValueError("max_tokens must be positive")
        self.layout, self.tables, self.embed_scale, self.grad_mode = layout, list(tables), float(embed_scale), grad_mode
        self.max_tokens, self.hidden, self.k_pad = max_tokens, weight.shape[0], info.k_pad
        # columns of ids that each table serves
        self.table_cols = info.cols if per_site else info.heads
        dev, seg = weight.device, info.seg_pitch
        T, h, K = max_tokens, self.hidden, self.k_pad
        kb, hb, tb = (-(-n // 128) for n in (K, h, T))
        held = torch.float32 if scales == "f32" else torch.uint8

        def codes(rows, blocks):
            return torch.empty((rows, 128 * blocks), dtype=torch.float8_e4m3fn, device=dev)

        def room(blocks, n):
            return torch.empty(blocks * n, dtype=held, device=dev)

        self.seg = seg
        self.rows = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
        self.rows_q, self.rows_s = codes(T, kb), room(kb, T)
        self.rows_t, self.rows_ts = codes(K, tb), room(tb, K)
        self.w_q, self.w_s = codes(h, kb), room(kb, hb).view(kb, hb)
        self.w_t, self.w_ts = codes(K, hb), room(hb, kb).view(hb, kb)
        self.v = torch.empty((T, h), dtype=torch.float32, device=dev)
        self.dv = torch.empty((T, h), dtype=torch.float32, device=dev)
        self.dv_q, self.dv_s = codes(T, hb), room(hb, T)
        self.dv_t, self.dv_ts = codes(h, tb), room(tb, h)
        self.d_rows = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
        self.d_weight = torch.empty((h, K), dtype=torch.float32, device=dev)
        # what backward reads of a forward's arguments: copies, so that the caller may refill its own
        self.streams = torch.empty((T, hc_mult, h), dtype=torch.bfloat16, device=dev)  # as they were before the add
        self.ids = torch.empty((T, 3 * info.heads), dtype=torch.int32, device=dev)
        self.keep = torch.empty(T, dtype=torch.uint8, device=dev)
        places = T * self.table_cols
        if grad_mode == "sparse":
            self.table_grads = [torch.empty((places, info.row_dim), dtype=grad_dtype, device=dev) for _ in tables]
            self.unique = [torch.empty(places, dtype=torch.int32, device=dev) for _ in tables]
            self.count = [torch.empty(1, dtype=torch.int32, device=dev) for _ in tables]
        else:
            self.table_grads = [torch.zeros(t.shape, dtype=grad_dtype, device=dev) for t in tables]
            self.unique = self.count = [None] * len(tables)
        # the gradient's size serves every smaller call; the split of a product changes with its
        # shape: room for the largest it takes up to max_tokens
        sizes = [engram_embed_grad_workspace(places, max(t.shape[0] for t in tables), info.row_dim)]
        sizes += [max(engram_fp8_matmul_workspace(n, h, K), engram_fp8_matmul_workspace(n, K, h),
                      engram_fp8_matmul_workspace(h, K, n)) for n in range(1, T + 1)]
        self.work = torch.empty(max(sizes), dtype=torch.uint8, device=dev)
        self._pending = None
        if stream is not None:
            # the buffers belong to the current stream: its zeros, and what it still does to memory
            # that they take over, come before the first call on `stream`
            here = torch.cuda.current_stream(dev)
            with _on(stream):
                torch.cuda.current_stream(dev).wait_stream(here)
        self.load_weight(weight, stream=stream)

    def load_weight(self, weight, *, stream=None):
        """Takes a [hidden][k_pad] weight over as 8-bit codes, in both the forms its products read.
        A forward that waits for its backward is dropped: its gradients are those of the weight
        that is written over."""
        if tuple(weight.shape) != (self.hidden, self.k_pad):
            raise ValueError(f"weight must be {[self.hidden, self.k_pad]}")
        self._pending = None
        engram_fp8_quantize(weight, self.w_q, self.w_s, q_t=self.w_t, scales_t=self.w_ts, block_rows=128, stream=stream)

    def _table_ids(self, n, T):
        return self.ids[:T, n * self.table_cols:(n + 1) * self.table_cols]

    def forward(self, row_ids, streams, *, site: int = 0, keep=None, stream=None):
        """Adds the memory that row_ids (int32 [T][sites][3][H], engram_compress_hash) name into
        ``streams`` (bf16 [T][hc][hidden], in place) and keeps what backward needs: a copy of the
        site's ids, of keep (uint8 [T]) and of the streams, so that all three may be refilled.
        A forward that waits for its backward is dropped by the next."""
        T = streams.shape[0]
        if not 1 <= T <= self.max_tokens:
            raise ValueError(f"{T} tokens, construct with max_tokens for them (1 .. {self.max_tokens})")
        if tuple(streams.shape[1:]) != tuple(self.streams.shape[1:]):
            raise ValueError(f"streams must be [T]{list(self.streams.shape[1:])}")
        if not 0 <= site < self.layout.info.num_sites:
            raise ValueError("site out of range")
        info = self.layout.info
        if not row_ids.is_cuda or row_ids.dtype != torch.int32:
            raise TypeError("row_ids must be a device tensor of int32")
        ids = row_ids.view(T, info.num_sites, 3 * info.heads)[:, site]
        if keep is not None:
            _flat(keep, "keep", torch.uint8)
            if keep.numel() < T:
                raise ValueError("keep too small")
        kb, tb = self.k_pad_blocks, -(-T // 128)
        self._pending = None  # from here on the buffers of an earlier forward are written over
        with _on(stream):
            self.ids[:T].copy_(ids)
            if keep is not None:
                self.keep[:T].copy_(keep.view(-1)[:T])
                keep = self.keep
        width = self.table_cols * self.seg
        for n, table in enumerate(self.tables):
            engram_embed(table, self._table_ids(n, T), self.rows[:T, n * width:(n + 1) * width], scale=self.embed_scale,
                         seg_pitch=self.seg, stream=stream)
        engram_fp8_quantize(self.rows[:T], self.rows_q, self.rows_s[:kb * T].view(kb, T), q_t=self.rows_t,
                            scales_t=self.rows_ts[:tb * self.k_pad].view(tb, self.k_pad), stream=stream)
        engram_fp8_matmul(self.rows_q[:T], self.rows_s[:kb * T].view(kb, T), self.w_q, self.w_s, self.v[:T],
                          workspace=self.work, stream=stream)
        with _on(stream):
            self.streams[:T].copy_(streams)
        engram_gate_add(self.layout, self.v, streams, keep=keep, T=T, stream=stream)
        self._pending = (T, keep)
        return streams

    def backward(self, d_streams, *, stream=None):
        """From the gradient of the streams that forward left (bf16, replaced by the gradient of
        the streams it was given): ``d_weight`` and ``table_grads`` (with ``unique`` and ``count``
        when sparse).  One backward per forward."""
        if self._pending is None:
            raise RuntimeError("no forward is waiting for its backward")
        T, keep = self._pending
        if tuple(d_streams.shape) != (T,) + tuple(self.streams.shape[1:]):
            raise ValueError("d_streams must have the shape of the forward's streams")
        hb, tb = -(-self.hidden // 128), -(-T // 128)
        engram_gate_add_backward(self.v, self.streams[:T], d_streams, d_streams, self.dv, keep=keep, stream=stream)
        self._pending = None  # d_streams is replaced: what is left cannot be started again
        dvs, dvts = self.dv_s[:hb * T].view(hb, T), self.dv_ts[:tb * self.hidden].view(tb, self.hidden)
        engram_fp8_quantize(self.dv[:T], self.dv_q, dvs, q_t=self.dv_t, scales_t=dvts, stream=stream)
        engram_fp8_matmul(self.dv_q[:T], dvs, self.w_t, self.w_ts, self.d_rows[:T], workspace=self.work, stream=stream)
        engram_fp8_matmul(self.dv_t[:, :128 * tb], dvts, self.rows_t[:, :128 * tb],
                          self.rows_ts[:tb * self.k_pad].view(tb, self.k_pad), self.d_weight, workspace=self.work,
                          stream=stream)
        width = self.table_cols * self.seg
        for n, table in enumerate(self.tables):
            engram_embed_grad(self._table_ids(n, T), self.d_rows[:T, n * width:(n + 1) * width], self.table_grads[n],
                              rows=table.shape[0], scale=self.embed_scale, mode=self.grad_mode, seg_pitch=self.seg,
                              unique=self.unique[n], count=self.count[n], workspace=self.work, stream=stream)
        return d_streams

    @property
    def k_pad_blocks(self) -> int:
        return -(-self.k_pad // 128)


def _on(stream):
    """The context that puts torch's own operations on ``stream`` (None: the current one)."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(stream))
