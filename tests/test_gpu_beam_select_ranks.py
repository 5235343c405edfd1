"""Which candidates a selection takes, at every rank and the last one too: token, parent and done flag
against a reference that lists candidates past the cut."""
import numpy as np
import pytest
import torch

from test_gpu_serve_ops import SELECTS, run_select, select_inputs, select_reference, status

pytestmark = pytest.mark.gpu

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")
TYPES = [torch.bfloat16, torch.float32]
PAST = 64  # candidates listed behind the cut


def check_ranks(x, scores, done, end, n, dtype, **how):
    """A kernel's total is off by tol at most (its derivation: the exponentials' differences to the
    largest logit, up to 104 where exp leaves fp32's range, take 2.5 roundings of 2^-24 and 2 units;
    the fp32 sums of a lane, a wave and four waves 41), so two candidates can change places where
    their totals are within 2 tol; those of one beam never, whose order is by logit and token."""
    x = torch.as_tensor(x).to(dtype).double().numpy()
    G, K = scores.shape
    ref = select_reference(x, scores, done, end, n + PAST)
    tokens, parents, out, out_done = run_select(x, scores, done, end, n, dtype, **how)
    assert status() == 0
    finite = x[np.isfinite(x)]
    spread = min(104.0, float(finite.max() - finite.min())) if finite.size else 0.0
    tol = 2.0 ** -24 * (2.5 * spread + 2 + 41)
    for g in range(G):
        own = {b: [v for _, c, v in ref[g] if c == b] for b in range(K)}
        taken = {b: 0 for b in range(K)}
        totals = np.array([t for t, _, _ in ref[g]])
        for i in range(n):
            b, v = int(parents[g, i]), int(tokens[g, i])
            if i >= len(ref[g]):
                assert (v, b, out[g, i], out_done[g, i]) == (-1, -1, -np.inf, 0)
                continue
            assert 0 <= b < K, (g, i)
            # a beam's candidates come in its own order, none left out
            assert v == own[b][taken[b]], (g, i)
            taken[b] += 1
            t, want_b, want_v = ref[g][i]
            near = {ref[g][j][1] for j in np.flatnonzero(np.abs(totals - t) <= 2 * tol)}
            if len(near) == 1:
                assert (b, v) == (want_b, want_v), (g, i)
            else:
                assert b in near, (g, i)
            assert out_done[g, i] == int(v == end or (done is not None and done[g, b] != 0)), (g, i)
            assert abs(float(out[g, i]) - t) <= 2 * tol + 2.0 ** -24 * abs(t) * 1.01, (g, i)
    return tokens, parents, out, out_done


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G, K, V, n", SELECTS + [(9, 1, 129_280, 1), (300, 1, 4097, 1), (33, 4, 20_001, 1), (40, 8, 65_536, 8)])
def test_every_rank(G, K, V, n, dtype):
    x, scores = select_inputs(G * 17 + V, G, K, V)
    check_ranks(x, scores, None, min(V - 1, 3), n, dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("masked", [0.3, 0.999])
@pytest.mark.parametrize("n", [1, 7, 64])
def test_every_rank_of_masked_rows_and_ended_beams(n, masked, dtype):
    x, scores = select_inputs(n, 12, 5, 30_011, masked)
    done = (np.random.default_rng(n).random((12, 5)) < 0.3).astype(np.uint8)
    done[3] = 1
    scores[5, 1:] = -np.inf
    check_ranks(x, scores, done, 30_010, n, dtype)


def crowded(kind, seed, G, K, V, dtype):
    """Rows many of whose logits are equal or nearly so."""
    rng = np.random.default_rng(seed)
    x, scores = select_inputs(seed, G, K, V)
    if kind.startswith("mask"):  # a finite number stands for a masked token
        low = {"mask_lowest": torch.finfo(dtype).min, "mask_1e4": -1e4, "mask_zero": 0.0}[kind]
        x = np.where(rng.random(x.shape) < 20 / V, np.abs(x) + 1.0, low)
        x[0] = low                       # nothing is left of this row
        x[1, :] = low
        x[1, V - 1] = 1.0                # and one token of this
    elif kind == "flat":                 # a model that has learnt nothing yet
        x = -11.77 + 0.02 * rng.standard_normal(x.shape)
    elif kind == "near":                 # float32's first 16 bits are the same for all
        x = 5.0 + rng.integers(0, 1 << 14, x.shape) * 2.0 ** -21
    elif kind == "steps":                # few values, each many times
        x = np.floor(x)
    elif kind == "signed_zeros":
        x = np.where(rng.random(x.shape) < 0.5, -0.0, 0.0)
        x[:, V // 2] = 1.0
    elif kind == "zero_border":          # the smallest numbers on both sides of zero
        x = rng.integers(-3000, 3000, x.shape) * 2.0 ** -149 if dtype == torch.float32 else np.floor(x) * 2.0 ** -133
    elif kind == "highest":
        x = np.where(rng.random(x.shape) < 0.9, torch.finfo(dtype).max, 0.0)
    else:
        x = np.full_like(x, 1.25)
    return x, scores


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["mask_lowest", "mask_1e4", "mask_zero", "flat", "near", "steps", "signed_zeros", "zero_border",
                                  "highest", "equal"])
@pytest.mark.parametrize("G, K, V, n", [(2, 4, 129_280, 4), (3, 3, 4097, 64), (40, 4, 16_384, 16), (130, 8, 8193, 8), (1, 64, 9001, 64),
                                        (520, 2, 8192, 5)])
def test_every_rank_of_crowded_rows(G, K, V, n, kind, dtype):
    x, scores = crowded(kind, n, G, K, V, dtype)
    check_ranks(x, scores, None, -1, n, dtype)


def narrow(kind, seed, G, K, V, dtype):
    """Rows masked by a finite number but for few tokens, so that masked ones are among the n best."""
    x, scores = select_inputs(seed, G, K, V)
    keep = np.zeros(V, dtype=bool)
    keep[[V // 3] if kind.endswith("1") else [0, V // 2, V - 1]] = True
    x[:, ~keep] = torch.finfo(dtype).min if kind.startswith("lowest") else -1e4
    if kind == "1e4_same":  # the same total for every masked token of every beam
        x[:] = x[0]
        scores[:] = -1.0
    return x, scores


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("ended", [False, True])
@pytest.mark.parametrize("kind", ["lowest_1", "lowest_3", "1e4_1", "1e4_3", "1e4_same"])
@pytest.mark.parametrize("G, K, V, n", [(1, 4, 129_280, 8), (3, 8, 20_001, 64), (40, 8, 8193, 16), (2, 64, 9001, 64), (1, 64, 129_280, 64),
                                        (1, 1, 500_000, 64)])
def test_every_rank_of_narrow_choices(G, K, V, n, kind, ended, dtype):
    x, scores = narrow(kind, n, G, K, V, dtype)
    done = None
    if ended:
        done = (np.random.default_rng(V).random((G, K)) < 0.3).astype(np.uint8)
        scores[:, K // 2:] -= 3.0
    check_ranks(x, scores, done, V - 1 if ended else -1, n, dtype)


def event_time(call, passes=5):
    """The least of some passes, so that one that is held up does not count."""
    call()
    marks = [torch.cuda.Event(enable_timing=True) for _ in range(passes + 1)]
    torch.cuda.synchronize()
    marks[0].record()
    for m in marks[1:]:
        call()
        m.record()
    torch.cuda.synchronize()
    return min(a.elapsed_time(b) for a, b in zip(marks, marks[1:]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["mask_lowest", "mask_1e4", "flat", "near", "steps", "equal"])
def test_crowded_rows_are_not_read_once_a_candidate(kind, dtype):
    """Their pieces are in registers already: where the lists overflow, the bound is raised there.  (16
    candidates by 16 passes over memory took 20 times the ordinary rows' time; up to 33 counts of
    registers take a few times it at most.)"""
    G, K, V, n = 64, 8, 65_536, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((G * K, V), generator=g, device="cuda") * 2.5
    plain = x.to(dtype)
    if kind.startswith("mask"):
        keep = torch.rand(x.shape, generator=g, device="cuda") < 20 / V
        x = torch.where(keep, x, torch.finfo(dtype).min if kind == "mask_lowest" else -1e4)
    elif kind == "flat":
        x = -11.77 + 0.008 * x
    elif kind == "near":
        x = 5.0 + torch.randint(0, 1 << 14, x.shape, generator=g, device="cuda") * 2.0 ** -21
    elif kind == "steps":
        x = x.floor()
    else:
        x = torch.full_like(x, 1.25)
    crowd = x.to(dtype)
    scores = -torch.rand((G, K), generator=g, device="cuda")
    out = [torch.empty((G, n), dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.float32)]
    work = torch.empty(eng.engram_beam_select_workspace(G, K, V, n), dtype=torch.uint8, device="cuda")
    times = [event_time(lambda: eng.engram_beam_select(t, scores, *out, workspace=work)) for t in (plain, crowd)]
    assert status() == 0
    assert times[1] <= 8 * times[0], times


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G, K, V, n", [(1, 4, 129_280, 8), (64, 8, 65_536, 16), (1, 64, 129_280, 64)])
@pytest.mark.parametrize("mask", ["lowest", -1e4])
def test_narrow_choices_are_not_joined_one_by_one(mask, G, K, V, n, dtype):
    """One allowed token a row: totals of masked ones are equal and reach the join's bound.  (4 beams and
    8 candidates took 100 times the ordinary rows' time.)"""
    g = torch.Generator(device="cuda").manual_seed(1)
    plain = (torch.randn((G * K, V), generator=g, device="cuda") * 2.5).to(dtype)
    crowd = torch.full_like(plain, torch.finfo(dtype).min if mask == "lowest" else mask)
    crowd[:, 77] = plain[:, 77]
    scores = -torch.rand((G, K), generator=g, device="cuda")
    out = [torch.empty((G, n), dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.float32)]
    work = torch.empty(eng.engram_beam_select_workspace(G, K, V, n), dtype=torch.uint8, device="cuda")
    times = [event_time(lambda: eng.engram_beam_select(t, scores, *out, workspace=work)) for t in (plain, crowd)]
    assert status() == 0
    # (an event's time of a call this short holds some 10 us of its own)
    assert times[1] <= 8 * times[0] + 0.02, times


@pytest.mark.parametrize("dtype", TYPES)
def test_one_graph_of_ordinary_and_crowded_rows(dtype):
    """Captured with ordinary logits, replayed with others, on a stream of its own, with eager work
    between the replays."""
    G, K, V, n = 5, 4, 40_003, 8
    inputs = [select_inputs(1, G, K, V)[0]] + [crowded(kind, 2, G, K, V, dtype)[0] for kind in ("mask_lowest", "flat", "equal")]
    inputs += [narrow(kind, 3, G, K, V, dtype)[0] for kind in ("lowest_1", "1e4_3")] + [select_inputs(4, G, K, V)[0]]
    inputs = [torch.as_tensor(x, device="cuda").to(dtype) for x in inputs]
    scores = -torch.rand((G, K), device="cuda")
    work = torch.empty(eng.engram_beam_select_workspace(G, K, V, n), dtype=torch.uint8, device="cuda")

    def outputs():
        return [torch.empty((G, n), dtype=t, device="cuda") for t in (torch.int32, torch.int32, torch.float32)]

    want = []
    for x in inputs:
        want.append(outputs())
        eng.engram_beam_select(x, scores, *want[-1], workspace=work)
    logits, out = inputs[0].clone(), outputs()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        eng.engram_beam_select(logits, scores, *out, workspace=work)
    for i in (1, 0, 2, 3, 5, 4, 6, 1):
        logits.copy_(inputs[i])
        for o in out:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.randn(1000, device="cuda").sum().item()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want[i])), i
    assert status() == 0
