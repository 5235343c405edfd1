"""The serving operators run together, as a beam search uses them, against a search on the host that
keeps every beam's whole sequence: what a beam's pages hold, what its store slot holds, which
pages are free.  Also on other streams and in graphs that are replayed."""
import numpy as np
import pytest
import torch

import engram_inputs as ei
from engram_harness import DEV, Site
from test_gpu_serve_ops import select_reference, unpack

pytestmark = pytest.mark.gpu

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype, device="cuda")


class HostSearch:
    """Beams as lists of tokens; totals in 64 bits, rounded to float as the operator's are."""

    def __init__(self, prompts, K, end):
        self.K, self.end = K, end
        self.seqs = [[list(p)] for p in prompts]
        self.scores = [[np.float32(0)] for _ in prompts]
        self.done = [[0] for _ in prompts]

    def step(self, logits):
        """logits [requests][beams now][V] float64."""
        tokens = np.full((len(self.seqs), self.K), -1)
        parents = np.full((len(self.seqs), self.K), -1)
        for g, seqs in enumerate(self.seqs):
            scores = np.array([self.scores[g]], dtype=np.float32)
            done = np.array([self.done[g]], dtype=np.uint8) if len(seqs) > 1 else None
            ref = select_reference(logits[g], scores, done, self.end, self.K)[0]
            self.scores[g] = [np.float32(t) for t, _, _ in ref]
            self.done[g] = [int(v == self.end or self.done[g][b]) for _, b, v in ref]
            self.seqs[g] = [seqs[b] + [v] for _, b, v in ref]
            tokens[g, :len(ref)], parents[g, :len(ref)] = [v for *_, v in ref], [b for _, b, _ in ref]
        return tokens, parents


def check_pages(d, search, cache, upto):
    """Every beam's first `upto` positions, read through its block table, are its sequence's; the
    pages in use are those the tables name."""
    P = d.page_size
    tables, free = d.tables.cpu().numpy(), unpack(d.free.cpu(), d.num_pages)
    lens = d.lens.cpu().numpy()
    used = set()
    for g, seqs in enumerate(search.seqs):
        own = set()
        for b, seq in enumerate(seqs):
            row = tables[g * d.beams + b]
            assert lens[g * d.beams + b] == upto[g]
            n = int(upto[g])
            pages = row[:-(-n // P)]
            own |= set(pages.tolist())
            for layer in range(cache.shape[0]):
                got = cache[layer].cpu().numpy()[pages].reshape(-1)[:n]
                assert got.tolist() == [t * (layer + 1) for t in seq[:n]], (g, b)
            if n % P:
                others = [tables[g * d.beams + c][n // P] for c in range(len(seqs)) if c != b]
                assert row[n // P] not in others
        assert not own & used
        used |= own
    assert set(np.flatnonzero(~free).tolist()) == used


@pytest.mark.parametrize("G, K, P, V, steps, end", [(1, 1, 4, 50, 9, -1), (3, 4, 4, 97, 20, 5), (2, 8, 1, 300, 12, -1),
                                                    (5, 3, 16, 1000, 40, 7), (2, 16, 5, 64, 17, 3), (1, 64, 8, 200, 10, -1)])
def test_search_with_paged_caches(G, K, P, V, steps, end):
    rng = np.random.default_rng(G * 10 + K)
    lens = rng.integers(1, 4 * P, G)
    lens[0] = 2 * P  # a prompt that ends with its page
    prompts = [rng.integers(0, V, n).tolist() for n in lens]
    max_len = int(lens.max()) + steps
    pages = G * K * -(-max_len // P)
    cache = torch.full((2, pages, P), -1, dtype=torch.int32, device="cuda")
    d = eng.BeamDecode(None, requests=G, beams=K, max_len=max_len, page_size=P, vocab=V, end_token=end, caches=[cache])
    search = HostSearch(prompts, K, end)

    def write(tokens):
        for layer in range(2):
            cache[layer].view(-1)[d.token_slots[:tokens.numel()]] = tokens * (layer + 1)

    for wave in range(2):  # the second after everything was given back
        d.start(dev(lens), int(lens.sum()) + 3)
        assert d.cu_seqlens.tolist() == np.concatenate([[0], np.cumsum(lens)]).tolist()
        assert d.positions[:int(lens.sum())].tolist() == [i for n in lens for i in range(n)]
        assert d.token_slots[int(lens.sum()):].tolist() == [-1] * 3
        write(dev(np.concatenate(prompts)))
        x = rng.standard_normal((G, V)).astype(np.float32) * 2
        want, _ = search.step(x.astype(np.float64)[:, None])
        d.first(dev(x, torch.float32))
        assert np.array_equal(d.tokens.cpu(), want)
        check_pages(d, search, cache, lens)
        for i in range(1, steps):
            d.plan()
            live = d.tokens.view(-1).clone()
            write(live)
            x = rng.standard_normal((G, K, V)).astype(np.float32) * 2
            x[rng.random(x.shape) < 0.2] = -np.inf
            want, parents = search.step(x.astype(np.float64))
            d.select(dev(x.reshape(G * K, V), torch.float32))
            assert np.array_equal(d.tokens.cpu(), want) and np.array_equal(d.parents.cpu(), parents), i
            assert np.array_equal(d.done.cpu(), search.done), i
            np.testing.assert_allclose(d.scores.cpu(), search.scores, rtol=0, atol=2e-5 * (1 + i))
            search.scores = [list(s) for s in d.scores.cpu().numpy()]  # (totals are carried as floats)
            check_pages(d, search, cache, lens + i)
        d.finish()
        assert eng.engram_get_error() == 0
        assert unpack(d.free.cpu(), d.num_pages).all()
        search = HostSearch(prompts, K, end)


@pytest.mark.parametrize("table_dtype", ["fp8", "bf16"])
def test_search_with_the_memory_of_a_site(table_dtype):
    """Prefill, selection and single steps of a site: the store's slots and the looked-up rows are
    those of every beam's whole sequence.  (bf16 tables have no lookup in one launch.)"""
    cfg = ei.get_config("decode_tiny", table_dtype=table_dtype)
    rng = np.random.default_rng(11)
    G, K, P, V, steps = 5, 4, 4, cfg.vocab, 9
    lens = rng.integers(1, 12, G)
    prompts = [rng.integers(0, V, n).tolist() for n in lens]
    site = Site(cfg, max_tokens=int(lens.sum()) + G * K).site
    assert site.decode_lookup_supported == (table_dtype == "fp8")
    check = Site(cfg, max_tokens=2048).site
    d = eng.BeamDecode(site, requests=G, beams=K, max_len=64, page_size=P, vocab=V)
    search = HostSearch(prompts, K, -1)
    tid2eid, pad = site.tid2eid.cpu().numpy(), site.pad_eid

    d.start(dev(lens), int(lens.sum()))
    tokens = dev(np.concatenate(prompts))
    streams = ei.make_streams(cfg, tokens.numel(), DEV)
    alone = streams.clone()
    d.prefill(tokens, streams)
    check.forward(tokens, d.cu_seqlens, alone)
    assert torch.equal(streams.view(torch.int16), alone.view(torch.int16))
    x = rng.standard_normal((G, V)).astype(np.float32) * 3
    search.step(x.astype(np.float64)[:, None])
    d.first(dev(x, torch.float32))
    for i in range(1, steps):
        d.plan()
        streams = ei.make_streams(cfg, G * K, DEV, step=i)
        alone = streams.clone()
        d.step(streams)
        # the same tokens as the last of whole sequences
        whole = [s for seqs in search.seqs for s in seqs]
        cu = np.concatenate([[0], np.cumsum([len(s) for s in whole])])
        last = dev(cu[1:] - 1).long()
        check.hash(dev(np.concatenate(whole)), dev(cu))
        assert torch.equal(site.row_ids[:G * K], check.row_ids[last]), i
        full = ei.make_streams(cfg, int(cu[-1]), DEV, step=100)
        full[last] = alone
        check.forward(dev(np.concatenate(whole)), dev(cu), full)
        # (another number of tokens is another order of the projection's sums)
        torch.testing.assert_close(streams.float(), full[last].float(), rtol=2 ** -7, atol=1e-3)
        x = rng.standard_normal((G, K, V)).astype(np.float32) * 3
        want, _ = search.step(x.astype(np.float64))
        d.select(dev(x.reshape(G * K, V), torch.float32))
        assert np.array_equal(d.tokens.cpu(), want), i
        search.scores = [list(s) for s in d.scores.cpu().numpy()]
        slots, ids = d.slots.cpu().numpy(), d.store.ids().cpu().numpy()
        assert sorted(slots.reshape(-1).tolist()) == list(range(G * K))
        for g in range(G):
            for b in range(K):  # the store holds the sequence up to the token that was fed last
                tail = [pad] * 3 + [int(tid2eid[t]) for t in search.seqs[g][b][:-1]]
                assert ids[slots[g, b]].tolist() == tail[-3:], (i, g, b)
    d.finish()
    assert eng.engram_get_error() == 0


def test_beams_that_nothing_is_left_for():
    """A vocabulary smaller than the beams: beams without a token stay so, keep their slots and pages,
    and the memory takes them as dead positions."""
    cfg = ei.get_config("decode_tiny")
    G, K, V = 2, 4, 3
    site = Site(cfg, max_tokens=64).site
    d = eng.BeamDecode(site, requests=G, beams=K, max_len=16, page_size=2, vocab=V)
    d.start(dev([3, 4]), 7)
    d.prefill(dev([1, 2, 0, 2, 1, 0, 1]), ei.make_streams(cfg, 7, DEV))
    d.first(torch.zeros((G, V), device="cuda"))
    assert d.tokens.tolist() == [[0, 1, 2, -1]] * 2 and d.parents.tolist() == [[0, 0, 0, -1]] * 2
    for _ in range(3):
        d.plan()
        streams = ei.make_streams(cfg, G * K, DEV)
        before = streams.clone()
        none = (d.tokens.view(-1) < 0).nonzero().view(-1)
        d.step(streams)
        assert torch.equal(streams[none].view(torch.int16), before[none].view(torch.int16))
        d.select(torch.zeros((G * K, V), device="cuda"))
        assert sorted(d.slots.view(-1).tolist()) == list(range(G * K))
    assert (d.tokens >= 0).all() and eng.engram_get_error() == 0
    d.finish()
    assert unpack(d.free.cpu(), d.num_pages).all()


def test_pool_that_runs_out_leaves_the_beams_as_they_were():
    d = eng.BeamDecode(None, requests=2, beams=2, max_len=64, page_size=2, vocab=10, num_pages=7)
    d.start(dev([2, 3]), 5)  # 1 + 2 pages, and one for the second request's other beam
    d.first(torch.zeros((2, 10), device="cuda"))
    assert eng.engram_get_error() == 0
    d.plan()  # two more for the first request, whose beams begin a block
    assert eng.engram_get_error() == 0
    sure = torch.zeros((4, 10), device="cuda")
    sure[:, 3] = 50.0  # every beam goes on with its own token, so no page comes back
    d.select(sure)
    assert d.parents.tolist() == [[0, 1]] * 2
    d.plan()  # two for the second request, and one is left
    state = [t.clone() for t in (d.tables, d.free, d.lens)]
    assert eng.engram_get_error() == eng.ENGRAM_E_PAGES
    assert d.cu_seqlens.tolist() == [0] * 5 and d.token_slots.tolist() == [-1] * 4
    d.plan()
    assert eng.engram_get_error() == eng.ENGRAM_E_PAGES
    assert all(torch.equal(a, b) for a, b in zip(state, (d.tables, d.free, d.lens)))


@pytest.mark.parametrize("lens", [[1, 2], [4, 5], [9, 12]])
def test_prompts_that_are_given_up_leave_no_fault(lens):
    """finish right after start: full blocks of the prompts are named by every beam."""
    d = eng.BeamDecode(None, requests=2, beams=3, max_len=16, page_size=4, vocab=10)
    for _ in range(2):
        d.start(dev(lens), sum(lens))
        d.finish()
        assert eng.engram_get_error() == 0
        assert unpack(d.free.cpu(), d.num_pages).all()


def test_construction_refuses():
    ok = dict(requests=2, beams=2, max_len=8, page_size=2, vocab=10)
    for change in (dict(requests=0), dict(beams=0), dict(beams=65), dict(max_len=0), dict(page_size=0),
                   dict(requests=8193, beams=1)):
        with pytest.raises(ValueError):
            eng.BeamDecode(None, **dict(ok, **change))
    with pytest.raises(ValueError):
        eng.BeamDecode(None, caches=[torch.zeros((3, 2), device="cuda")], **ok)
    d = eng.BeamDecode(None, **ok)
    for lens, n in ((dev([1]), 2), (dev([1, 1], torch.int64), 2), (dev([1, 1]), 17), (dev([1, 1]), -1), (dev([1, 1]).cpu(), 2)):
        with pytest.raises(ValueError):
            d.start(lens, n)
    d.start(dev([1, 1]), 2)
    with pytest.raises(RuntimeError):
        d.start(dev([1, 1]), 2)
    d.finish()
    d.start(dev([1, 1]), 2)
    assert eng.engram_get_error() == 0


# ---------------------------------------------------------------------------
# streams and graphs
# ---------------------------------------------------------------------------

def test_steps_on_another_stream_and_in_a_graph():
    """A whole step, captured once and replayed with new logits, equals the same steps run eagerly, with
    eager work between the replays; and so do steps on a stream of their own."""
    G, K, P, V, steps = 6, 4, 2, 5003, 12
    g = torch.Generator(device="cuda").manual_seed(3)
    first = torch.randn((G, V), generator=g, device="cuda")
    x = [torch.randn((G * K, V), generator=g, device="cuda") for _ in range(steps)]
    lens = dev([1, 2, 3, 4, 5, 6])

    def begin(stream=None):
        cache = torch.arange(2 * G * K * 16 * P, device="cuda", dtype=torch.int32).view(2, G * K * 16, P)
        d = eng.BeamDecode(None, requests=G, beams=K, max_len=16 * P, page_size=P, vocab=V, end_token=4, caches=[cache])
        torch.cuda.synchronize()
        d.start(lens, 21, stream=stream)
        d.first(first, stream=stream)
        return d, cache

    def state(d, cache):
        return [t.clone() for t in (d.tokens, d.parents, d.scores, d.done, d.slots, d.lens, d.tables, d.free, d.page_src,
                                    d.page_dst, d.token_slots, d.positions, d.cu_seqlens, cache)]

    want = []
    d, cache = begin()
    for logits in x:
        d.plan()
        d.select(logits)
        want.append(state(d, cache))
    assert eng.engram_get_error() == 0

    side = torch.cuda.Stream()
    d, cache = begin(side)
    for logits, w in zip(x, want):
        d.plan(stream=side)
        d.select(logits, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(state(d, cache), w))
    assert eng.engram_get_error(side) == 0

    d, cache = begin()
    logits = x[0].clone()
    d.plan()  # (what a captured call needs before it is captured)
    d.select(logits)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d.plan()
        d.select(logits)
    for i in range(1, steps):
        logits.copy_(x[i])
        graph.replay()
        torch.randn(1000, device="cuda").sum().item()
        assert all(torch.equal(a, b) for a, b in zip(state(d, cache), want[i])), i
    assert eng.engram_get_error() == 0


def test_a_busy_current_stream_is_waited_for_only_where_it_is_needed():
    """Made for another stream: buffers are filled before its first call.  Lengths that are a strided
    view are made contiguous on the call's stream, not behind what the current one still does."""
    def state(d):
        return [t.clone() for t in (d.tokens, d.parents, d.scores, d.slots, d.lens, d.tables, d.free, d.token_slots,
                                    d.positions, d.cu_seqlens, d.seq_start)]

    size = dict(requests=3, beams=2, max_len=64, page_size=4, vocab=1000)
    logits = torch.randn((3, 1000), device="cuda")
    lens = dev([5, 99, 8, 99, 3, 99])[::2]
    work = torch.ones((8192, 8192), device="cuda")
    d = eng.BeamDecode(None, **size)
    d.start(lens, 16)
    d.first(logits)
    want = state(d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        work @ work
    d = eng.BeamDecode(None, stream=side, **size)
    side.synchronize()
    for _ in range(4):
        work @ work
    d.start(lens, 16, stream=side)
    d.first(logits, stream=side)
    with torch.cuda.stream(side):
        got = state(d)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert eng.engram_get_error(side) == 0


def test_selections_at_the_same_time():
    """Two streams, a workspace each."""
    G, K, V, n = 8, 4, 40_000, 8
    cases = []
    for seed in range(2):
        g = torch.Generator(device="cuda").manual_seed(seed)
        logits = torch.randn((G * K, V), generator=g, device="cuda")
        scores = -torch.rand((G, K), generator=g, device="cuda")
        out = [torch.empty((G, n), dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.float32)]
        work = torch.empty(eng.engram_beam_select_workspace(G, K, V, n), dtype=torch.uint8, device="cuda")
        eng.engram_beam_select(logits, scores, *out, workspace=work)
        cases.append((logits, scores, [o.clone() for o in out], out, work, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for o in (o for c in cases for o in c[3]):
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for logits, scores, _, out, work, stream in cases:
            eng.engram_beam_select(logits, scores, *out, workspace=work, stream=stream)
    torch.cuda.synchronize()
    for _, _, want, out, *_ in cases:
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_selection_workspace_serves_smaller_calls():
    V, n = 30_000, 5
    work = torch.empty(eng.engram_beam_select_workspace(50, 8, V, n), dtype=torch.uint8, device="cuda")
    logits = torch.randn((400, V), device="cuda")
    scores = -torch.rand((50, 8), device="cuda")
    full = None
    for G in (50, 17, 4, 1):
        out = [torch.empty((G, n), dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.float32)]
        eng.engram_beam_select(logits[:8 * G], scores[:G], *out, workspace=work)
        if full is None:
            full = out
        assert torch.equal(out[0], full[0][:G]) and torch.equal(out[1], full[1][:G])
        torch.testing.assert_close(out[2], full[2][:G], rtol=0, atol=1e-5)
    assert eng.engram_get_error() == 0
