"""Calls of SiteTraining beside one whole step: sizes between, buffers that change, calls that fail."""
import pytest
import torch

from test_gpu_training import BF16, DEV, eng, make  # noqa: F401  (eng is a fixture)

pytestmark = pytest.mark.gpu


def step(site, row_ids, x, dy, T, **kw):
    """One forward and backward of the first T tokens: everything they leave."""
    y, d = x[:T].clone(), dy[:T].clone()
    site.forward(row_ids[:T], y, **kw)
    site.backward(d)
    n = [int(c) for c in site.count]
    return [y, d, site.d_weight.clone()] + [g[:c].clone() for g, c in zip(site.table_grads, n)] + \
        [u[:c].clone() for u, c in zip(site.unique, n)]


@pytest.mark.parametrize("T", [1297, 1365, 1400])
def test_every_call_up_to_max_tokens(eng, T):
    """24 x 256 columns: the gradient of 1,365 tokens takes more scratch than that of 1,400."""
    L, tables, w, site, row_ids, x, dy, _ = make(eng, per_site=True, T=1400, row_dim=256, heads=8)
    own = eng.SiteTraining(L, tables, w, max_tokens=T, embed_scale=0.5)
    for a, b in zip(step(site, row_ids, x, dy, T), step(own, row_ids, x, dy, T)):
        assert torch.equal(a, b)
    assert eng.engram_get_error() == 0


@pytest.mark.parametrize("sites, mode", [(1, "sparse"), (2, "accumulate")])
def test_backward_after_the_callers_buffers_are_refilled(eng, sites, mode):
    """row_ids, keep and streams of the forward hold the next call's values by the time of backward."""
    L, tables, w, site, row_ids, x, dy, keep = make(eng, per_site=False, sites=sites, mode=mode)
    other = eng.SiteTraining(L, tables, w, max_tokens=150, embed_scale=0.5, grad_mode=mode)
    left = []
    for s, refill in ((site, False), (other, True)):
        ids, k, y, d = row_ids.clone(), keep.clone(), x.clone(), dy.clone()
        s.forward(ids, y, site=sites - 1, keep=k)
        if refill:
            ids.copy_(ids.flip(0))
            k.copy_(1 - k)
            y.zero_()
        s.backward(d)
        torch.cuda.synchronize()
        n = [int(c) if c is not None else t.shape[0] for c, t in zip(s.count, s.table_grads)]
        left.append([d, s.d_weight, s.dv] + [g[:c] for g, c in zip(s.table_grads, n)])
    for a, b in zip(*left):
        assert torch.equal(a, b)


def test_forward_refuses_ids_and_masks_it_would_convert(eng):
    L, tables, w, site, row_ids, x, dy, keep = make(eng, per_site=True)
    with pytest.raises(TypeError):
        site.forward(row_ids.long(), x.clone())
    with pytest.raises(TypeError):
        site.forward(row_ids.cpu(), x.clone())
    with pytest.raises(TypeError):
        site.forward(row_ids, x.clone(), keep=keep.bool())
    with pytest.raises(ValueError):
        site.forward(row_ids, x.clone(), keep=keep[:20])


def test_a_forward_that_fails_leaves_nothing_for_backward(eng):
    """Streams of the wrong type are turned down by the gate, behind the projection: the buffers no
    longer hold the forward before, and there is no backward of it."""
    L, tables, w, site, row_ids, x, dy, keep = make(eng, per_site=True)
    site.forward(row_ids, x.clone())
    with pytest.raises(TypeError):
        site.forward(row_ids.flip(0), x.float())
    with pytest.raises(RuntimeError):
        site.backward(dy.clone())
    # arguments that are turned down before anything is written leave it waiting
    y, want = dy.clone(), dy.clone()
    site.forward(row_ids, x.clone())
    with pytest.raises(ValueError):
        site.forward(row_ids, x.clone(), site=1)
    with pytest.raises(TypeError):
        site.backward(dy.float())
    site.backward(y)
    other = eng.SiteTraining(L, tables, w, max_tokens=150, embed_scale=0.5)
    other.forward(row_ids, x.clone())
    other.backward(want)
    assert torch.equal(y, want)


def test_a_backward_that_fails_cannot_be_started_again(eng):
    """What fails behind the gate's gradient has replaced d_streams: a second run would apply it twice."""
    L, tables, w, site, row_ids, x, dy, keep = make(eng, per_site=True)
    site.forward(row_ids, x.clone())
    work, site.work = site.work, site.work[:0]
    d = dy.clone()
    with pytest.raises(eng.EngramError):
        site.backward(d)
    site.work = work
    with pytest.raises(RuntimeError):
        site.backward(d)


def test_a_new_weight_drops_the_forward_of_the_old_one(eng):
    """backward multiplies by the weight of its forward, which load_weight writes over."""
    L, tables, w, site, row_ids, x, dy, keep = make(eng, per_site=True)
    site.forward(row_ids, x.clone())
    site.load_weight(w * 2)
    with pytest.raises(RuntimeError):
        site.backward(dy.clone())


def test_construction_for_another_stream(eng):
    """The current stream is still busy when the site is made: the weight it writes and the zeros of
    the gradients come before what the site does on its stream."""
    L, tables, w, plain, row_ids, x, dy, keep = make(eng, per_site=False, mode="accumulate")
    side, ready, late = torch.cuda.Stream(), w.clone(), torch.zeros_like(w)
    got, want = (x.clone(), dy.clone()), (x.clone(), dy.clone())
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)  # some 20 ms
    late.copy_(ready)
    site = eng.SiteTraining(L, tables, late, max_tokens=150, embed_scale=0.5, grad_mode="accumulate", stream=side)
    site.forward(row_ids, got[0], stream=side)
    site.backward(got[1], stream=side)
    torch.cuda.synchronize()
    plain.forward(row_ids, want[0])
    plain.backward(want[1])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(site.d_weight, plain.d_weight)
    for a, b in zip(site.table_grads, plain.table_grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("sites", [1, 2])
def test_a_captured_step_replays_with_new_inputs(eng, sites):
    """Forward and backward in one graph; every replay, after the inputs were refilled, against the same
    calls made eagerly."""
    L, tables, w, site, row_ids, x, dy, keep = make(eng, per_site=False, sites=sites, mode="accumulate")
    other = eng.SiteTraining(L, tables, w, max_tokens=150, embed_scale=0.5, grad_mode="accumulate")
    ids, k, y, d = row_ids.clone(), keep.clone(), x.clone(), dy.clone()

    def run(s):
        s.forward(ids, y, site=sites - 1, keep=k)
        s.backward(d)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(site)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(site)
    for turn in range(4):
        left = []
        for s, go in ((site, graph.replay), (other, lambda: run(other))):
            ids.copy_(row_ids.roll(7 * turn, 0))
            k.copy_(keep.roll(turn, 0))
            y.copy_(x.roll(turn, 0))
            d.copy_(dy.roll(3 * turn, 0))
            for t in s.table_grads:
                t.zero_()
            go()
            torch.cuda.synchronize()
            left.append([t.clone() for t in (y, d, s.d_weight, *s.table_grads)])
        for a, b in zip(*left):
            assert torch.equal(a, b), turn
