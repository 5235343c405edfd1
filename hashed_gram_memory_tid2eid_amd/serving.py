"""Beam decoding around an Engram site runner: the serving operators chained over preallocated
device buffers, with no host synchronisation.

``BeamDecode`` keeps, for ``requests`` requests of ``beams`` beams each, what a decode loop
carries from step to step: slots of the n-gram memory's rolling store, block tables over a pool
of pages, lengths, total scores and which beams have ended.  The order of a step follows the
pages' generation graph, sampler -> n-gram memory -> backbone ([VeOmni#1370] "feat: support
DeepSeek-V4.1-Flash in SeedOmni", generate commit); pages and slots are those that a backbone
keeps its caches in ([vLLM-V41] "vllm/models/deepseek_v41/nvidia/model",
DeepseekV4Model.__init__: the hash state is keyed by the KV cache's slots).

    d = BeamDecode(engram, requests=G, beams=K, max_len=4096, page_size=16, vocab=V, end_token=2, caches=[kv])
    d.start(lens, num_tokens)           # pages of the prompts: d.cu_seqlens, d.token_slots, d.positions
    d.prefill(tokens, streams)          # the n-gram memory of the prompts
    ...                                 # the model, whose cache rows are d.token_slots
    d.first(logits)                     # [G][V] at the prompts' last tokens: every request's K beams
    for _ in range(d.max_len - longest):  # at most, until all of d.done
        d.plan()                        # a place for one more token a beam
        d.step(streams)                 # the n-gram memory of d.tokens
        ...                             # the model
        d.select(logits)                # [G * K][V]: d.tokens, d.parents, d.scores, d.done
    d.finish()                          # every page is free again
"""
from __future__ import annotations

from . import (engram_beam_reorder, engram_beam_select, engram_beam_select_workspace, engram_block_plan,
               engram_block_release, engram_state_copy)


class BeamDecode:
    """State of ``requests`` x ``beams`` decoding beams on the current device.

    ``engram``: the site runner whose store the beams use, or None for selection and block tables
    alone.  ``caches``: tensors [pages][width] or [layers][pages][width] whose rows are the pool's
    pages; they are copied where beams part inside a page.  ``num_pages`` defaults to a whole
    table for every beam; it may be less, since the beams of a request share what they have in
    common.  ``stream``: that of the first calls, behind all that the current stream holds.
    ``max_len``: tokens of a beam, prompt and all, rounded up to whole pages: the attribute max_len
    is what plan keeps to, and what a model's positions have to reach.

    All requests go on together, ended ones too (they take a place a step until finish), and plan
    refuses every beam where one would pass max_len: take it for the longest prompt and all steps.

    Buffers on the device: tokens, parents, slots, scores, done [requests][beams]; lens and tables,
    a row a beam; free, the pool.  Of the last plan: cu_seqlens, seq_start, token_slots and
    positions.  parents and tokens are overwritten by every selection: a caller that wants the
    whole sequences keeps them.  Faults that only the device sees latch as everywhere
    (engram_get_error)."""

    def __init__(self, engram, *, requests: int, beams: int, max_len: int, page_size: int, vocab: int, end_token: int = -1,
                 num_pages=None, caches=(), max_prompt_tokens=None, stream=None):
        import torch
        if requests < 1 or not 1 <= beams <= 64 or max_len < 1 or page_size < 1:
            raise ValueError("requests, max_len and page_size must be positive, beams 1 to 64")
        if not -1 <= end_token < vocab:
            raise ValueError("end_token must be a token of the vocabulary, or -1")
        G, K, n = requests, beams, requests * beams
        if n > 8192:
            raise ValueError("at most 8,192 beams in all")
        if engram is not None and engram.max_tokens < n:
            raise ValueError(f"{n} beams > the runner's max_tokens {engram.max_tokens}")
        self.engram, self.requests, self.beams, self.page_size = engram, G, K, page_size
        self.blocks = -(-max_len // page_size)
        self.max_len = self.blocks * page_size
        self.num_pages = n * self.blocks if num_pages is None else int(num_pages)
        self.end_token, self.caches = end_token, list(caches)
        self.max_prompt_tokens = G * self.max_len if max_prompt_tokens is None else int(max_prompt_tokens)
        places = max(self.max_prompt_tokens, n)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.store = None if engram is None else engram.make_store(n, stream=stream)
        self.slots = torch.arange(n, **i32).view(G, K)
        self.tables = torch.full((n, self.blocks), -1, **i32)
        self.lens = torch.zeros(n, **i32)
        bits = torch.arange(-(-self.num_pages // 32) * 32, device="cuda").view(-1, 32) < self.num_pages
        self.free = (bits.long() << torch.arange(32, device="cuda")).sum(1).to(torch.uint32).view(torch.int32)
        self.tokens, self.parents, self.page_src, self.page_dst = (torch.zeros((G, K), **i32) for _ in range(4))
        for c in self.caches:
            # a copy of no row, whose refusals would otherwise come at the first selection, when
            # the beams have moved
            engram_state_copy(c, self.page_src, self.page_dst)
            if c.shape[-2] < self.num_pages:
                raise ValueError("a cache has fewer pages than the pool")
        self.scores = torch.zeros((G, K), dtype=torch.float32, device="cuda")
        self.done = torch.zeros((G, K), dtype=torch.uint8, device="cuda")
        self.seq_start = torch.zeros(n, dtype=torch.uint8, device="cuda")
        self._cu, self._past, self._new, self._ones = (torch.full((n + 1,), i, **i32) for i in (0, 0, 0, 1))
        self._token_slots = torch.full((places,), -1, dtype=torch.int64, device="cuda")
        self._positions = torch.zeros(places, **i32)
        # the plan that gives the other beams a last page each: its tokens are the prompt's own
        self._tail_cu = torch.zeros(n + 1, **i32)
        self._tail_slots = torch.empty(G * (K - 1) * (page_size - 1), dtype=torch.int64, device="cuda")
        self._prompt_scores = torch.zeros((G, 1), dtype=torch.float32, device="cuda")
        self._work = torch.empty(max(engram_beam_select_workspace(G, 1, vocab, K),
                                     engram_beam_select_workspace(G, K, vocab, K)), dtype=torch.uint8, device="cuda")
        self._all = torch.ones(n, dtype=torch.uint8, device="cuda")
        self._none = torch.zeros(n, dtype=torch.uint8, device="cuda")
        self._each = torch.arange(n + 1, **i32)
        self._started = False
        self._rows_planned(0, 0)
        if stream is not None:
            # the buffers belong to the current stream: what it fills them with comes before the
            # first call on `stream`
            here = torch.cuda.current_stream()
            with _on(stream):
                torch.cuda.current_stream().wait_stream(here)

    def _rows_planned(self, rows, tokens):
        self.cu_seqlens = self._cu[:rows + 1]
        self.token_slots, self.positions = self._token_slots[:tokens], self._positions[:tokens]

    def start(self, lens, num_tokens: int, *, stream=None):
        """Pages for prompts of ``lens`` int32 [requests] tokens, each at least one, held by every
        request's first beam, and a last page for each of its other beams.  num_tokens: places
        for the prompts' tokens, at least their sum.  Afterwards cu_seqlens [requests + 1],
        token_slots, positions and seq_start are those of the prompts.  A fault is latched: prompts
        that do not fit (their pages, num_tokens, max_len) take nothing and every length is 0;
        where only the last pages do not fit, the first beams hold the prompts and the others
        their full blocks.  finish follows either way."""
        import torch
        G, K, P = self.requests, self.beams, self.page_size
        if self._started:
            raise RuntimeError("the last prompts' beams still hold their pages: call finish first")
        if tuple(lens.shape) != (G,) or lens.dtype != torch.int32 or not lens.is_cuda:
            raise ValueError("lens must be int32 [requests] on the device")
        if not 0 <= num_tokens <= self.max_prompt_tokens:
            raise ValueError(f"{num_tokens} tokens, max_prompt_tokens is {self.max_prompt_tokens}")
        self._started = True
        pool = dict(page_size=P, num_pages=self.num_pages, stream=stream)
        with _on(stream):
            self.lens.zero_()
            self.done.zero_()
            held, lens = self.lens.view(G, K)[:, 0].contiguous(), lens.contiguous()
        self._rows_planned(G, num_tokens)
        engram_block_plan(held, lens, self.tables.view(G, K * self.blocks)[:, :self.blocks], self.free,
                          cu_seqlens=self.cu_seqlens, token_slots=self.token_slots, positions=self.positions,
                          seq_start=self.seq_start[:G], lens=held, **pool)
        with _on(stream):
            # from here on the lengths that were granted: 0 after a fault, when the tables still
            # name pages of earlier prompts
            past, new = self._past[:G * K].view(G, K), self._new[:G * K].view(G, K)
            new.zero_()
            if K > 1:
                new[:, 1:] = held.remainder(P)[:, None]
            past.copy_(held[:, None]).sub_(new)
            # the other beams name the prompt's blocks, too, so that finish may follow at once
            tables = self.tables.view(G, K, self.blocks)
            tables[:, 1:] = tables[:, :1]
        engram_block_plan(self._past[:G * K], self._new[:G * K], self.tables, self.free, cu_seqlens=self._tail_cu,
                          token_slots=self._tail_slots, lens=self.lens, **pool)

    def prefill(self, tokens, streams, *, dead=None, keep=None, stream=None):
        """The n-gram memory of the prompts (int32, one after another) added into streams, and
        their tails into the first beams' slots."""
        with _on(stream):
            slots = self.slots[:, 0].contiguous()
        return self.engram.forward(tokens, self.cu_seqlens, streams, seq_start=self.seq_start[:self.requests], slots=slots,
                                   store=self.store, dead=dead, keep=keep, stream=stream)

    def first(self, logits, *, stream=None):
        """The first tokens: every request's ``beams`` best of logits [requests][vocab] at its
        prompt's last token; all beams continue the first one."""
        engram_beam_select(logits, self._prompt_scores, self.tokens, self.parents, self.scores, workspace=self._work,
                           done_out=self.done, end_token=self.end_token, stream=stream)
        self._follow(stream)

    def plan(self, *, stream=None):
        """A place for one more token of every beam: cu_seqlens [n + 1], token_slots, positions
        and seq_start, row by row.  A beam that passes max_len, or a pool without pages, latches
        its fault and leaves everything as it was."""
        n = self.requests * self.beams
        self._rows_planned(n, n)
        engram_block_plan(self.lens, self._ones[:n], self.tables, self.free, page_size=self.page_size,
                          num_pages=self.num_pages, cu_seqlens=self.cu_seqlens, token_slots=self.token_slots,
                          positions=self.positions, seq_start=self.seq_start, lens=self.lens, stream=stream)

    def step(self, streams, *, stream=None):
        """The n-gram memory of the selected tokens added into streams [requests * beams][hc][hidden]
        (several sites: one such tensor each).  A beam without a token (none was left to select)
        counts as dead."""
        import torch
        with _on(stream):
            flat = self.tokens.view(-1)
            dead, keep = (flat < 0).to(torch.uint8), (flat >= 0).to(torch.uint8)
        args = dict(slots=self.slots.view(-1), store=self.store, dead=dead, keep=keep, stream=stream)
        if self.engram.decode_lookup_supported:
            return self.engram.decode_step(flat, streams, **args)
        return self.engram.forward(flat, self._each, streams, seq_start=self._none, **args)

    def select(self, logits, *, stream=None):
        """The next tokens from logits [requests * beams][vocab] of the last ones; slots, store,
        tables and caches follow the selected beams."""
        engram_beam_select(logits, self.scores, self.tokens, self.parents, self.scores, workspace=self._work,
                           done=self.done if self.end_token >= 0 else None, done_out=self.done, end_token=self.end_token,
                           stream=stream)
        self._follow(stream)

    def _follow(self, stream):
        engram_beam_reorder(self.parents, slots=self.slots, store=self.store, tables=self.tables, lens=self.lens,
                            page_size=self.page_size, num_pages=self.num_pages, free=self.free, page_src=self.page_src,
                            page_dst=self.page_dst, stream=stream)
        for c in self.caches:
            engram_state_copy(c, self.page_src, self.page_dst, stream=stream)

    def finish(self, *, stream=None):
        """Every beam's pages are free again, and the next prompts may start."""
        engram_block_release(self.tables, self.lens, self._all, self.free, page_size=self.page_size,
                             num_pages=self.num_pages, stream=stream)
        with _on(stream):
            self.lens.zero_()
        self._started = False


def _on(stream):
    """The small tensor operations of a call, on its stream."""
    import contextlib
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    return torch.cuda.stream(stream)
