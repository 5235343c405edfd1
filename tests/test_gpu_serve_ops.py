"""The serving operators on the GPU against plain implementations: loops over Python integers for
block tables, slots and reordering (all compared exactly), 64-bit floats for the selection."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")
I32, I64, U8 = torch.int32, torch.int64, torch.uint8


def dev(x, dtype=I32):
    return torch.as_tensor(x, dtype=dtype, device="cuda")


def status():
    return eng.engram_get_error()


# ---------------------------------------------------------------------------
# pools
# ---------------------------------------------------------------------------

def pack(bits):
    wide = np.zeros(-(-len(bits) // 32) * 32, dtype=np.uint8)
    wide[:len(bits)] = bits
    return np.packbits(wide, bitorder="little").view(np.int32).copy()


def unpack(words, n):
    return np.unpackbits(np.asarray(words, dtype=np.int32).view(np.uint8), bitorder="little")[:n].astype(bool)


def blocks_of(n, P):
    return -(-int(n) // P)


def random_rows(rng, R, blocks, P, past, spare):
    """Tables of rows with these lengths over a pool with `spare` pages left, and the pool's bits."""
    held = sum(blocks_of(p, P) for p in past)
    num_pages = held + spare
    pages = rng.permutation(num_pages)
    tables = np.full((R, blocks), -1, dtype=np.int32)
    at = 0
    for r in range(R):
        n = blocks_of(past[r], P)
        tables[r, :n] = pages[at:at + n]
        at += n
    free = np.zeros(num_pages, dtype=bool)
    free[pages[held:]] = True
    return tables, free, num_pages


def plan_reference(past, new, tables, free, P, T):
    """(cu, start, lens, positions, slots, tables, free) as Python integers give them."""
    tables, free = tables.copy(), free.copy()
    pages = iter(np.flatnonzero(free))
    cu, positions, slots = [0], [], []
    for r, (p, n) in enumerate(zip(past, new)):
        for b in range(blocks_of(p, P), blocks_of(p + n, P)):
            tables[r, b] = next(pages)
            free[tables[r, b]] = False
        for pos in range(p, p + n):
            positions.append(pos)
            slots.append(int(tables[r, pos // P]) * P + pos % P)
        cu.append(cu[-1] + n)
    rest = T - cu[-1]
    return (cu, [int(p == 0) for p in past], [p + n for p, n in zip(past, new)], positions + [0] * rest, slots + [-1] * rest,
            tables, free)


def run_plan(past, new, tables, free, num_pages, P, T, *, apart=False, alias=False, pad=0):
    """The call's outputs as numpy arrays, in plan_reference's order."""
    R = len(past)
    wide = dev(np.concatenate([tables, np.full((R, pad), 77, dtype=np.int32)], 1))
    t = wide[:, :tables.shape[1]]
    words = dev(pack(free))
    out = torch.full_like(words, -1) if apart else None
    p, n = dev(past), dev(new)
    lens = p if alias else torch.full((R,), -5, dtype=I32, device="cuda")
    cu, start = torch.full((R + 1,), -5, dtype=I32, device="cuda"), torch.full((R,), 9, dtype=U8, device="cuda")
    positions, slots = torch.full((T,), -5, dtype=I32, device="cuda"), torch.full((T,), -5, dtype=I64, device="cuda")
    eng.engram_block_plan(p, n, t, words, page_size=P, num_pages=num_pages, cu_seqlens=cu, token_slots=slots,
                          positions=positions, seq_start=start, lens=lens, free_out=out)
    got = [x.cpu().numpy() for x in (cu, start, lens, positions, slots, t, words if out is None else out)]
    assert (wide[:, tables.shape[1]:] == 77).all()
    if apart:
        assert (words.cpu().numpy() == pack(free)).all()
    got[6] = unpack(got[6], num_pages)
    return got


PLANS = [  # R, P, most blocks a row, most new tokens a row, spare pages, padding of T
    (1, 16, 4, 1, 3, 0), (1, 1, 5, 5, 40, 7), (2, 16, 3, 40, 100, 0), (63, 16, 9, 1, 64, 1), (64, 64, 5, 1, 2000, 0),
    (65, 7, 12, 30, 3000, 100), (255, 16, 17, 2, 300, 1), (256, 16, 32, 1, 5000, 0), (257, 3, 9, 20, 3000, 0),
    (1023, 16, 6, 1, 1100, 1), (1024, 5, 7, 3, 2000, 0), (1025, 32, 3, 1, 1100, 31), (4097, 16, 4, 1, 5000, 0),
    (8192, 16, 3, 1, 9000, 0), (3, 256, 40, 9000, 200, 5), (17, 16, 200, 900, 2000, 0), (40, 100, 60, 4000, 70_000, 3),
]


@pytest.mark.parametrize("how", ["in_place", "apart", "alias", "strided"])
@pytest.mark.parametrize("R, P, blocks, most, spare, pad", PLANS)
def test_plan(R, P, blocks, most, spare, pad, how):
    rng = np.random.default_rng(R * 1000 + P)
    new = rng.integers(0, most + 1, R)
    new = np.minimum(new, blocks * P)
    past = (rng.random(R) * (blocks * P - new + 1)).astype(np.int64) * (rng.random(R) < 0.8)
    need = sum(blocks_of(p + n, P) - blocks_of(p, P) for p, n in zip(past, new))
    tables, free, num_pages = random_rows(rng, R, blocks, P, past, max(spare, need))
    T = int(new.sum()) + pad
    want = plan_reference(past.tolist(), new.tolist(), tables, free, P, T)
    got = run_plan(past, new, tables, free, num_pages, P, T, apart=how == "apart", alias=how == "alias",
                   pad=5 if how == "strided" else 0)
    assert status() == 0
    for name, g, w in zip(("cu", "start", "lens", "positions", "slots", "tables", "free"), got, want):
        assert np.array_equal(g, np.asarray(w)), name


@pytest.mark.parametrize("num_pages", [1, 31, 32, 33, 8192, 32_768, 262_144, 262_145, 1_000_003])
@pytest.mark.parametrize("where", ["first", "last", "every", "sparse"])
def test_plan_takes_the_lowest_free_pages(num_pages, where):
    rng = np.random.default_rng(num_pages)
    free = np.zeros(num_pages, dtype=bool)
    if where == "first":
        free[:max(1, num_pages // 2)] = True
    elif where == "last":
        free[-max(1, num_pages // 7):] = True
    elif where == "every":
        free[:] = True
    else:
        free[rng.choice(num_pages, max(1, num_pages // 50), replace=False)] = True
    for take in sorted({1, min(5, int(free.sum())), min(3000, int(free.sum()))}):
        tables = np.full((1, take), -1, dtype=np.int32)
        want = plan_reference([0], [take], tables, free, 1, take)
        got = run_plan([0], [take], tables, free, num_pages, 1, take)
        assert status() == 0
        assert np.array_equal(got[5], want[5]) and np.array_equal(got[6], want[6])
        assert np.array_equal(got[4], want[4])


@pytest.mark.parametrize("num_pages", [20_000, 262_144, 300_000, 2_000_003])
@pytest.mark.parametrize("R", [1, 37, 1025, 8192])
@pytest.mark.parametrize("density", [0.02, 0.5, 1.0])
def test_plan_of_many_pages(num_pages, R, density):
    """More pages than are looked for one by one, for rows with many, with one and with none."""
    rng = np.random.default_rng(R + num_pages)
    free = rng.random(num_pages) < density
    total = min(int(free.sum()), 17_000)
    cut = np.sort(rng.integers(0, total + 1, R - 1))
    new = np.diff(np.concatenate([[0], cut, [total]]))
    blocks = int(new.max()) + 3
    past = rng.integers(0, 4, R)
    tables = np.full((R, blocks), -1, dtype=np.int32)
    for take in {True, total < int(free.sum())}:  # exactly what there is, or some are left
        some = free.copy()
        if take:
            some[np.flatnonzero(free)[total:]] = False
        tables[:] = -1
        want = plan_reference(past.tolist(), new.tolist(), tables, some, 1, total + 1)
        got = run_plan(past, new, tables, some, num_pages, 1, total + 1, apart=not take)
        assert status() == 0
        for name, g, w in zip(("cu", "start", "lens", "positions", "slots", "tables", "free"), got, want):
            assert np.array_equal(g, np.asarray(w)), name


def test_plan_leaves_bits_behind_the_pool():
    words = dev([-1, -1])
    t = torch.full((1, 40), -1, dtype=I32, device="cuda")
    cu, slots = torch.zeros(2, dtype=I32, device="cuda"), torch.zeros(40, dtype=I64, device="cuda")
    eng.engram_block_plan(dev([0]), dev([40]), t, words, page_size=1, num_pages=40, cu_seqlens=cu, token_slots=slots)
    assert status() == 0
    assert words.tolist() == [0, -256] and t[0].tolist() == list(range(40)) == slots.tolist()


def test_plan_of_no_rows_and_of_no_tokens():
    e = torch.zeros(0, dtype=I32, device="cuda")
    cu, slots = torch.full((1,), 9, dtype=I32, device="cuda"), torch.zeros(3, dtype=I64, device="cuda")
    eng.engram_block_plan(e, e, e.view(0, 4), dev([7]), page_size=4, num_pages=3, cu_seqlens=cu, token_slots=slots)
    assert cu.tolist() == [0] and slots.tolist() == [-1] * 3
    cu = torch.full((3,), 9, dtype=I32, device="cuda")
    eng.engram_block_plan(dev([5, 0]), dev([0, 0]), dev([[2, 1], [-1, -1]]), dev([1]), page_size=4, num_pages=3, cu_seqlens=cu,
                          token_slots=slots[:0])
    assert cu.tolist() == [0, 0, 0] and status() == 0


def test_plan_slots_pass_32_bits():
    pages = (1 << 30) - 1
    t = dev([[pages - 1, -1]])
    cu, slots = torch.zeros(2, dtype=I32, device="cuda"), torch.zeros(2, dtype=I64, device="cuda")
    words = torch.zeros(1 << 25, dtype=I32, device="cuda")
    words[-1] = 1 << 5
    eng.engram_block_plan(dev([255]), dev([2]), t, words, page_size=256, num_pages=pages, cu_seqlens=cu, token_slots=slots)
    last = 32 * ((1 << 25) - 1) + 5
    assert status() == 0 and t[0].tolist() == [pages - 1, last]
    assert slots.tolist() == [(pages - 1) * 256 + 255, last * 256] and int(words[-1]) == 0


@pytest.mark.parametrize("T", [8, 5000])
@pytest.mark.parametrize("past, new, spare, code", [
    ([3, -1], [1, 1], 4, "SEQLENS"), ([3, 3], [1, -1], 4, "SEQLENS"), ([3, 16], [1, 1], 4, "SEQLENS"),
    ([0, 0], [5000, 1], 4, "SEQLENS"), ([3, 2147483647], [1, 2147483647], 4, "SEQLENS"), ([8, 4], [1, 4], 1, "PAGES"),
    ([0, 0], [4, 4], 0, "PAGES"),
])
def test_plan_that_does_not_fit_takes_nothing(past, new, spare, code, T):
    ok = [p if 0 <= p <= 16 else 0 for p in past]
    tables, free, num_pages = random_rows(np.random.default_rng(1), 2, 4, 4, ok, spare)
    got = run_plan(past, new, tables, free, num_pages, 4, T)
    assert status() == eng.STATUS["ENGRAM_E_" + code]
    assert got[0].tolist() == [0, 0, 0] and got[2].tolist() == list(past) and (got[4] == -1).all() and (got[3] == 0).all()
    assert np.array_equal(got[5], tables) and np.array_equal(got[6], free)


@pytest.mark.parametrize("T", [7, 4999, 40])
def test_plan_of_more_tokens_than_places(T):
    past, new = np.zeros(3, dtype=np.int64), np.array([T, 0, 1])
    tables, free, num_pages = random_rows(np.random.default_rng(2), 3, 400, 16, past, 700)
    got = run_plan(past, new, tables, free, num_pages, 16, T, apart=True)
    assert status() == eng.ENGRAM_E_SEQLENS
    assert got[0].tolist() == [0] * 4 and (got[4] == -1).all() and np.array_equal(got[6], free)


@pytest.mark.parametrize("page", [-1, 9, 1 << 30])
def test_plan_reports_a_page_outside_the_pool(page):
    for T in (4, 5000):
        got = run_plan([2], [4], np.array([[page, -1]], dtype=np.int32), np.array([False] * 8 + [True]), 9, 4, T)
        assert status() == eng.ENGRAM_E_PAGE_RANGE
        assert got[4][:4].tolist() == [-1, -1, 32, 33] and got[0].tolist() == [0, 4]


@pytest.mark.parametrize("R, blocks, P", [(1, 1, 1), (3, 300, 16), (256, 40, 16), (5000, 3, 5), (2, 5000, 2)])
def test_release(R, blocks, P):
    rng = np.random.default_rng(R + blocks)
    lens = rng.integers(0, blocks * P + 1, R)
    tables, free, num_pages = random_rows(rng, R, blocks, P, lens, 17)
    if R > 2:  # two rows that share what they have
        lens[1] = lens[0]
        tables[1] = tables[0]
    flags = (rng.random(R) < 0.5).astype(np.uint8) * 3
    want = free.copy()
    for r in range(R):
        if flags[r]:
            want[tables[r, :blocks_of(lens[r], P)]] = True
    words = dev(pack(free))
    wide = dev(np.concatenate([tables, np.full((R, 3), 1 << 30, dtype=np.int32)], 1))
    for _ in range(2):  # a page given back twice is free
        eng.engram_block_release(wide[:, :blocks], dev(lens), dev(flags, U8), words, page_size=P, num_pages=num_pages)
    assert status() == 0
    assert np.array_equal(unpack(words.cpu(), num_pages), want)


def test_release_leaves_what_is_wrong():
    tables = dev([[0, 1], [2, 40], [3, 4], [5, -1]])
    words = dev([0])
    eng.engram_block_release(tables, dev([9, 8, -1, 8]), dev([1, 1, 1, 1], U8), words, page_size=4, num_pages=30)
    assert status() in (eng.ENGRAM_E_SEQLENS, eng.ENGRAM_E_PAGE_RANGE)
    assert words.tolist() == [1 << 2 | 1 << 5]


# ---------------------------------------------------------------------------
# selection
# ---------------------------------------------------------------------------

def select_reference(x, scores, done, end, n):
    """Per request the list of (total, beam, token) in order, totals in 64 bits."""
    G, K = scores.shape
    V = x.shape[1]
    out = []
    for g in range(G):
        totals, beams, logits, tokens = [], [], [], []
        for b in range(K):
            score, row = np.float64(scores[g, b]), x[g * K + b]
            if not np.isfinite(score):
                continue
            if done is not None and done[g, b]:
                totals.append([score]), beams.append([b]), logits.append([0.0]), tokens.append([end])
                continue
            if np.isnan(row).any() or (row == np.inf).any() or not np.isfinite(row).any():
                continue
            most = row.max()
            with np.errstate(under="ignore"):
                norm = math.log(np.exp(row - most).sum())
            live = np.flatnonzero(row > -np.inf)
            if len(live) > n:  # no more than n of a beam are among the n largest
                live = live[np.argsort(-row[live], kind="stable")[:n]]
            totals.append((score + (row[live] - most)) - norm), beams.append([b] * len(live))
            logits.append(row[live]), tokens.append(live)
        if totals:
            t, b, l, v = (np.concatenate([np.asarray(p, dtype=np.float64) for p in q]) for q in (totals, beams, logits, tokens))
            order = np.lexsort((v, -l, b, -t))[:n]
            out.append([(t[i], int(b[i]), int(v[i])) for i in order])
        else:
            out.append([])
    return out


def run_select(x, scores, done, end, n, dtype, *, ld=None, offset=0, in_place=False):
    G, K = scores.shape
    V = x.shape[1]
    ld = V if ld is None else ld
    flat = torch.full((offset + G * K * ld + 8,), float("nan"), dtype=dtype, device="cuda")
    logits = torch.as_strided(flat, (G * K, V), (ld, 1), offset)
    logits.copy_(torch.as_tensor(x, device="cuda").to(dtype))
    s, d = dev(scores, torch.float32), None if done is None else dev(done, U8)
    tokens, parents = (torch.full((G, n), -7, dtype=I32, device="cuda") for _ in range(2))
    out = s if in_place else torch.full((G, n), 5.0, device="cuda")
    out_done = d if in_place and d is not None else torch.full((G, n), 9, dtype=U8, device="cuda")
    work = torch.full((eng.engram_beam_select_workspace(G, K, V, n),), 0xA5, dtype=U8, device="cuda")
    eng.engram_beam_select(logits, s, tokens, parents, out, done=d, done_out=out_done, end_token=end, workspace=work)
    return [t.cpu().numpy() for t in (tokens, parents, out, out_done)]


def check_select(x, scores, done, end, n, dtype, **how):
    """Totals: a rounding to float (2^-24) of score + (x - most) - norm, where norm's error is that of
    the exponentials: a difference to the largest logit and its product with log2(e) are rounded
    (2^-24 |x - most| each at most, the constant's 2^-26 and the unit of the exponential itself
    beside them: under 2.5 x 2^-24 |x - most| + 2 x 2^-24), and of the fp32 sums of one lane (at
    most 32 terms an accumulator), its two accumulators, a wave (6 steps) and four waves (2):
    41 x 2^-24.  All terms are positive, so norm
    is off by their weighted mean, at most by the largest.  |x - most| counts at most to 104, where
    exp leaves fp32's range."""
    x = torch.as_tensor(x).to(dtype).double().numpy()
    want = select_reference(x, scores, done, end, n)
    tokens, parents, out, out_done = run_select(x, scores, done, end, n, dtype, **how)
    assert status() == 0
    finite = x[np.isfinite(x)]
    spread = min(104.0, float(finite.max() - finite.min())) if finite.size else 0.0
    tol = 2.0 ** -24 * (2.5 * spread + 2 + 41)
    for g in range(scores.shape[0]):
        ref = want[g]
        for i in range(n):
            if i >= len(ref):
                assert (tokens[g, i], parents[g, i], out[g, i], out_done[g, i]) == (-1, -1, -np.inf, 0)
                continue
            t, b, v = ref[i]
            near = [r for r in ref if abs(r[0] - t) <= 2 * tol]
            mine = (int(parents[g, i]), int(tokens[g, i]))
            if all(r[1] == b for r in near) and (i + 1 < n or len(ref) < n):
                assert mine == (b, v), (g, i)
            elif i + 1 < n:  # another beam's total is as near as the sums are exact
                assert mine in [(r[1], r[2]) for r in near], (g, i)
            assert abs(float(out[g, i]) - t) <= tol + 2.0 ** -24 * abs(t) * 1.01, (g, i)
            ended = mine[1] == end or (done is not None and how.get("in_place") is not True and bool(done[g, mine[0]]))
            if not how.get("in_place"):
                assert out_done[g, i] == int(ended)
        names = [(int(p), int(v)) for p, v in zip(parents[g], tokens[g]) if p >= 0]
        assert len(set(names)) == len(names)
    return tokens, parents, out, out_done


def select_inputs(seed, G, K, V, masked=0.0, std=2.5):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((G * K, V)) * std
    x[rng.random(x.shape) < masked] = -np.inf
    return x, -np.cumsum(rng.random((G, K)), 1).astype(np.float32)


SELECTS = [(1, 1, 1, 1), (1, 1, 1, 4), (1, 1, 7, 64), (1, 4, 1000, 4), (2, 3, 2047, 5), (2, 4, 2048, 8), (2, 4, 2049, 8),
           (3, 5, 4097, 10), (5, 2, 16_384, 4), (3, 8, 32_003, 16), (1, 4, 129_280, 4), (1, 1, 129_280, 64), (2, 64, 1000, 64),
           (1, 64, 9001, 64), (7, 8, 129_280, 8), (40, 8, 30_011, 16), (130, 8, 8193, 8), (300, 1, 513, 2), (64, 1, 65_537, 33)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G, K, V, n", SELECTS)
def test_select(G, K, V, n, dtype):
    x, scores = select_inputs(G * 31 + V, G, K, V)
    check_select(x, scores, None, -1, n, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [0, 1, 3, 8])
@pytest.mark.parametrize("extra", [0, 1, 24])
def test_select_rows_anywhere(offset, extra, dtype):
    """Rows that start inside a 16-byte line; NaN between them."""
    x, scores = select_inputs(offset, 3, 4, 5003)
    check_select(x, scores, None, 5, 8, dtype, ld=5003 + extra, offset=offset)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("masked", [0.5, 0.99, 0.9999])
def test_select_masked_and_done(masked, dtype):
    x, scores = select_inputs(int(masked * 10_000), 9, 6, 20_011, masked)
    rng = np.random.default_rng(3)
    done = (rng.random((9, 6)) < 0.3).astype(np.uint8)
    scores[1] = -np.inf
    scores[2, 1:] = -np.inf
    scores[3, 0], scores[3, 1], scores[3, 2] = np.nan, np.inf, 0.0
    done[4] = 1
    x[5 * 6:5 * 6 + 2] = -np.inf
    check_select(x, scores, done, 20_010, 12, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_rows_without_a_distribution(dtype):
    x, scores = select_inputs(8, 4, 3, 3001)
    x[0, 17] = np.nan
    x[1, 2999] = np.inf
    x[4, :] = np.nan
    x[5, 5], x[5, 6] = np.inf, -np.inf
    x[6:9, 100] = np.nan  # a request with nothing left
    x[9, :] = np.inf
    check_select(x, scores, None, -1, 6, dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V, n", [(3, 8), (70, 4), (5000, 16), (129_280, 8)])
def test_select_equal_logits(V, n, dtype):
    """Equal logits go by token, equal totals by beam, also where lists of candidates overflow."""
    x = np.full((6, V), 1.25)
    scores = np.zeros((2, 3), dtype=np.float32)
    scores[1] = (-1.0, 0.0, 0.0)
    tokens, parents, _, _ = check_select(x, scores, None, -1, n, dtype)
    for g in range(2):
        order = [(b, v) for b in ((0, 1, 2) if g == 0 else (1, 2, 0)) for v in range(V)][:n]
        assert [(int(p), int(v)) for p, v in zip(parents[g], tokens[g])][:len(order)] == order
    few = np.where(np.arange(V) % 3 == 1, 2.0, -1.0) + np.zeros((6, 1))
    tokens, parents, _, _ = check_select(few, scores, None, -1, n, dtype)
    first = [v for v in range(V) if v % 3 == 1][:n]
    assert tokens[0][:len(first)].tolist() == first and (parents[0][:len(first)] == 0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("G, K, V, n", [(1, 64, 5000, 64), (300, 1, 32_768, 3), (1, 64, 64, 64)])
def test_select_equal_logits_past_every_list(G, K, V, n, dtype):
    """More equal candidates than the lists of a piece, of its loads and of a request hold."""
    x = np.zeros((G * K, V))
    scores = np.zeros((G, K), dtype=np.float32)
    tokens, parents, *_ = check_select(x, scores, None, -1, n, dtype)
    assert (tokens == np.arange(n)).all() and (parents == 0).all()
    scores[:, ::2] = -1.0
    done = np.zeros((G, K), dtype=np.uint8)
    done[:, -1] = 1  # an ended beam's one candidate, the best of all
    scores[:, -1] = 1.0
    if K > 1:
        tokens, parents, *_ = check_select(x, scores, done, V - 1, n, dtype)
        assert (tokens[:, 0] == V - 1).all() and (parents[:, 0] == K - 1).all()
        assert (tokens[:, 1:] == np.arange(n - 1)).all() and (parents[:, 1:] == 1).all()


def test_select_zeros_of_both_signs_are_equal():
    x = np.zeros((1, 600))
    x[0, ::2] = -0.0
    for dtype in (torch.bfloat16, torch.float32):
        tokens, *_ = check_select(x, np.zeros((1, 1), dtype=np.float32), None, -1, 5, dtype)
        assert tokens[0].tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_select_lowest_values_and_wide_ranges(dtype):
    low = torch.finfo(dtype).min
    x, scores = select_inputs(4, 3, 2, 4001)
    x[0] = low               # a row masked by the type's lowest value all through: every token alike
    x[1, 10:] = low
    x[2, 5:] = low
    x[2, :5] = 3e38
    x[3] = np.linspace(-200.0, 200.0, 4001)
    x[4, :] = -np.inf
    x[4, 777] = low
    tokens, parents, out, _ = check_select(x, scores, None, -1, 7, dtype)
    assert [int(v) for p, v in zip(parents[2], tokens[2]) if p == 0] == [777]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("offset", [-1000.0, 700.0, 1023.0, 1025.0, 4097.0, 3e4, -1e5, 1e6, 3e8, -2e12, 1e20, 1e37])
def test_select_logits_far_from_zero(offset, dtype):
    """exp(x - most) where logits are large and their differences are not (float32 keeps fewer of them;
    bf16 keeps few that differ at all)."""
    x, scores = select_inputs(12, 3, 4, 20_001)
    check_select(x + offset, scores, None, -1, 8, dtype)


@pytest.mark.parametrize("V", [4096, 129_280])
def test_select_pieces_of_different_sizes(V):
    """Pieces whose maxima are far apart, on both sides of where exponents are taken differently."""
    x, scores = select_inputs(13, 2, 3, V)
    x[:, : V // 2] += 1030.0
    x[1, : V // 4] -= 3000.0
    x[2, V // 3:] -= 1e30
    check_select(x, scores, None, -1, 8, torch.float32)


def test_select_orders_a_beam_by_its_logits():
    """Steps of float32's last bit, in rising and falling order, with a list that starts full."""
    base = np.float32(7.0)
    steps = base + np.arange(3000, dtype=np.float32) * np.float32(2.0 ** -21)
    for x in (steps, steps[::-1].copy()):
        tokens, *_ = check_select(x[None].astype(np.float64), np.zeros((1, 1), dtype=np.float32), None, -1, 20, torch.float32)
        want = np.argsort(-x, kind="stable")[:20]
        assert tokens[0].tolist() == want.tolist()


def test_select_in_place():
    x, scores = select_inputs(6, 5, 4, 3000)
    done = np.zeros((5, 4), dtype=np.uint8)
    done[:, 1] = 1
    apart = check_select(x, scores, done, 9, 4, torch.float32)
    again = check_select(x, scores, done, 9, 4, torch.float32, in_place=True)
    for a, b in zip(apart, again):
        assert np.array_equal(a, b)


# ---------------------------------------------------------------------------
# reordering
# ---------------------------------------------------------------------------

def assign(parents):
    """(heir, continued) of every child of one request's beams."""
    K = len(parents)
    seen, heir = set(), [None] * K
    for c, p in enumerate(parents):
        if p >= 0 and p not in seen:
            seen.add(p)
            heir[c] = p
    spare = iter(b for b in range(K) if b not in seen)
    heir = [next(spare) if h is None else h for h in heir]
    return heir, [p if p >= 0 else h for p, h in zip(parents, heir)]


def reorder_reference(parents, slots, tables, lens, free, P):
    G, K = parents.shape
    tables_out, free = tables.copy(), free.copy()
    slots_out, pairs, pages = np.empty_like(slots), np.full((2, G, K), -1), np.full((2, G, K), -1)
    for g in range(G):
        heir, cont = assign(parents[g].tolist())
        L = int(lens[g * K])
        full = L // P
        old = tables[g * K:(g + 1) * K]
        for c in range(K):
            slots_out[g, c] = slots[g, heir[c]]
            row = tables_out[g * K + c]
            row[:full] = old[cont[c], :full]
            if L % P:
                row[full] = old[heir[c], full]
            if heir[c] != cont[c]:
                if slots[g, heir[c]] >= 0 and slots[g, cont[c]] >= 0:
                    pairs[:, g, c] = slots[g, cont[c]], slots[g, heir[c]]
                if L % P:
                    pages[:, g, c] = old[cont[c], full], old[heir[c], full]
        gone = set(old[:, :full].ravel().tolist()) - set(tables_out[g * K:(g + 1) * K, :full].ravel().tolist())
        for page in gone - {-1}:
            free[page] = True
    return slots_out, pairs, tables_out, pages, free


def beams_with_history(rng, G, K, blocks, P):
    """Tables as a search leaves them: shared blocks that split, every partly filled page its own."""
    num_pages = G * K * blocks + 5
    pages = rng.permutation(num_pages)
    tables = np.full((G * K, blocks), -1, dtype=np.int32)
    lens = np.repeat(rng.integers(0, blocks * P + 1, G), K)
    at = 0
    for g in range(G):
        L = int(lens[g * K])
        line = np.zeros(K, dtype=np.int64)  # which beams share the block
        for b in range(blocks_of(L, P)):
            if b * P + P > L:
                line = np.arange(K)
            elif rng.random() < 0.3:
                line = np.where(rng.random(K) < 0.3, np.arange(K), line)
            for i in sorted(set(line.tolist())):
                tables[g * K:(g + 1) * K, b][line == i] = pages[at]
                at += 1
    free = np.ones(num_pages, dtype=bool)
    free[tables[tables >= 0]] = False
    return tables, lens.astype(np.int32), free, num_pages


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("G, K, blocks, P", [(1, 1, 3, 16), (1, 4, 5, 16), (3, 2, 1, 1), (7, 5, 300, 7), (2, 8, 600, 16),
                                             (64, 8, 20, 16), (2, 64, 257, 3), (3, 33, 40, 5), (200, 3, 2, 2), (1, 16, 256, 4)])
def test_reorder(G, K, blocks, P, in_place):
    rng = np.random.default_rng(G * 100 + K)
    tables, lens, free, num_pages = beams_with_history(rng, G, K, blocks, P)
    parents = rng.integers(0, K, (G, K))
    parents[rng.random((G, K)) < 0.1] = -1
    if G > 2:
        parents[0] = np.arange(K)
        parents[1] = 0
        parents[2] = -1
    slots = rng.permutation(G * K + 3)[:G * K].reshape(G, K)
    if K > 2:
        slots[0, 1] = -1
    want = reorder_reference(parents, slots, tables, lens, free, P)
    t, s, words = dev(np.concatenate([tables, np.full((G * K, 2), 9, dtype=np.int32)], 1)), dev(slots), dev(pack(free))
    t_out = t if in_place else t.clone()
    s_out = s if in_place else torch.empty_like(s)
    pairs = [torch.full((G, K), 99, dtype=I32, device="cuda") for _ in range(4)]
    eng.engram_beam_reorder(dev(parents), slots=s, slots_out=s_out, slot_src=pairs[0], slot_dst=pairs[1], tables=t[:, :blocks],
                            tables_out=t_out[:, :blocks], lens=dev(lens), page_size=P, num_pages=num_pages, free=words,
                            page_src=pairs[2], page_dst=pairs[3])
    assert status() == 0
    assert np.array_equal(s_out.cpu(), want[0]) and np.array_equal(t_out.cpu()[:, :blocks], want[2])
    assert (t_out[:, blocks:] == 9).all()
    for i in range(2):
        assert np.array_equal(pairs[i].cpu(), want[1][i]) and np.array_equal(pairs[2 + i].cpu(), want[3][i])
    assert np.array_equal(unpack(words.cpu(), num_pages), want[4])
    if not in_place:
        assert np.array_equal(t.cpu()[:, :blocks], tables) and np.array_equal(s.cpu(), slots)


def small_store(slots):
    layout = eng.engram_layout_create(vocab_size=100, compressed_vocab=50, pad_token_id=0, heads_per_order=1, rows=[1000] * 3,
                                      row_dim=64, table_dtype=eng.ENGRAM_DTYPE_BF16, row_pitch_bytes=128)
    ids = torch.arange(3 * slots, dtype=I32, device="cuda").view(slots, 3) % 50
    return eng.engram_store_create(layout, 0, slots, ids=ids), ids.cpu().numpy()


@pytest.mark.parametrize("G, K", [(1, 1), (5, 4), (3, 64)])
def test_reorder_copies_store_entries(G, K):
    rng = np.random.default_rng(K)
    store, ids = small_store(G * K + 4)
    parents = rng.integers(-1, K, (G, K))
    slots = rng.permutation(G * K + 4)[:G * K].reshape(G, K)
    s = dev(slots)
    eng.engram_beam_reorder(dev(parents), slots=s, store=store)
    assert status() == 0
    got, want = store.ids().cpu().numpy(), ids.copy()
    for g in range(G):
        heir, cont = assign(parents[g].tolist())
        for c in range(K):
            want[slots[g, heir[c]]] = ids[slots[g, cont[c]]]
            assert int(s[g, c]) == slots[g, heir[c]]
    assert np.array_equal(got, want)


def test_reorder_leaves_what_is_wrong():
    tables = dev([[0, 1], [0, 2], [3, 4], [3, 5]])
    before = tables.clone()
    slots = dev([[0, 1], [2, 3]])
    words, pairs = dev([0]), [torch.zeros((2, 2), dtype=I32, device="cuda") for _ in range(4)]

    def go(parents, lens, num_pages=6):
        eng.engram_beam_reorder(dev(parents), slots=slots, slot_src=pairs[0], slot_dst=pairs[1], tables=tables, lens=dev(lens),
                                page_size=4, num_pages=num_pages, free=words, page_src=pairs[2], page_dst=pairs[3])

    for bad in (2, -2, 1 << 30):
        go([[bad, 0], [0, 1]], [6] * 4)
        assert status() == eng.ENGRAM_E_PARENT_RANGE
    for lens in ([6, 7, 6, 6], [9, 9, 6, 6], [-1, -1, 6, 6]):
        go([[0, 0], [0, 1]], lens)
        assert status() == eng.ENGRAM_E_SEQLENS
    assert torch.equal(tables, before) and slots.tolist() == [[0, 1], [2, 3]] and words.tolist() == [0]
    assert all((p == -1).all() for p in pairs)
    go([[0, 0], [0, 1]], [6] * 4, num_pages=2)  # the page to copy to is outside the pool
    assert status() == eng.ENGRAM_E_PAGE_RANGE
    assert all((p == -1).all() for p in pairs[2:])
    tables.copy_(dev([[0, 1], [0, 70], [3, 4], [3, 5]]))
    go([[0, 0], [0, 1]], [8] * 4)  # so is a page to free
    assert status() == eng.ENGRAM_E_PAGE_RANGE and words.tolist() == [0]
    store, ids = small_store(4)
    eng.engram_beam_reorder(dev([[0, 0]]), slots=dev([[1, 4]]), store=store)
    assert status() == eng.ENGRAM_E_SLOT_RANGE and np.array_equal(store.ids().cpu(), ids)


# ---------------------------------------------------------------------------
# copies
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("planes, rows, width, dtype, n", [
    (1, 2, 1, torch.uint8, 1), (1, 10, 3, I32, 4), (3, 17, 5, torch.uint8, 8), (2, 9, 4096, torch.bfloat16, 4),
    (5, 33, 1000, torch.bfloat16, 16), (1, 300, 12, torch.float32, 140), (2, 8, 100_003, torch.uint8, 3),
    (32, 20, 8192, torch.bfloat16, 9), (1, 70_000, 4, I32, 33_000), (2, 5, 70_000, I64, 2), (1, 4, 65, torch.float16, 2),
])
@pytest.mark.parametrize("pad", [0, 1])
def test_copy(planes, rows, width, dtype, n, pad):
    rng = np.random.default_rng(width)
    raw = torch.as_tensor(rng.integers(0, 256, (planes, rows, (width + pad) * torch.empty(0, dtype=dtype).element_size()),
                                       dtype=np.uint8)).cuda()
    state = raw.view(dtype)[:, :, :width]
    order = rng.permutation(rows)
    dst, src = order[:n].copy(), order[n:][rng.integers(0, rows - n, n)]
    dst[rng.random(n) < 0.2] = -1
    src[rng.random(n) < 0.2] = -1
    want = raw.cpu().numpy().copy()
    size = width * state.element_size()
    for s, d in zip(src, dst):
        if s >= 0 and d >= 0:
            want[:, d, :size] = want[:, s, :size]
    eng.engram_state_copy(state if planes > 1 else state[0], dev(src), dev(dst))
    assert status() == 0
    assert np.array_equal(raw.cpu().numpy(), want)


def test_copy_of_interleaved_planes():
    state = torch.arange(6 * 4 * 8, dtype=I32, device="cuda").view(6, 4, 8)  # [rows][planes][width]
    want = state.clone()
    want[5] = want[1]
    eng.engram_state_copy(state.transpose(0, 1), dev([1, 2]), dev([5, 2]))
    assert torch.equal(state, want) and status() == 0
    with pytest.raises(ValueError):
        eng.engram_state_copy(state[:1].expand(3, 4, 8), dev([1]), dev([2]))


@pytest.mark.parametrize("shape, strides, good", [((2, 4, 8), (4, 32, 1), False), ((2, 4, 8), (8, 15, 1), False),
                                                  ((2, 4, 8), (31, 8, 1), False), ((2, 4, 8), (8, 16, 1), True),
                                                  ((2, 4, 8), (32, 8, 1), True), ((2, 4, 8), (9, 17, 1), True)])
def test_copy_takes_planes_that_do_not_overlap(shape, strides, good):
    state = torch.zeros(256, dtype=I32, device="cuda").as_strided(shape, strides)
    if good:
        state[:, 1] = 5
        eng.engram_state_copy(state, dev([1]), dev([2]))
        assert (state[:, 1:3] == 5).all() and int(state.sum()) == 160 and status() == 0
    else:
        with pytest.raises(ValueError):
            eng.engram_state_copy(state, dev([1]), dev([2]))


def test_copy_skips_rows_that_are_not_there():
    state = torch.arange(12, device="cuda", dtype=I32).view(3, 4)
    want = state.clone()
    want[2] = want[0]
    eng.engram_state_copy(state, dev([0, 3, 0, -2]), dev([2, 1, 1 << 30, 1]))
    assert status() == eng.ENGRAM_E_SLOT_RANGE and torch.equal(state, want)


def test_copy_passes_32_bits():
    state = torch.zeros((5, 1 << 20, 1024), dtype=U8, device="cuda")  # 5 GiB
    state[:, 7] = 3
    eng.engram_state_copy(state, dev([7]), dev([(1 << 20) - 1]))
    assert status() == 0
    assert (state[:, -1] == 3).all() and int(state[:, -2].sum()) == 0 and int(state[4, 0].sum()) == 0


# ---------------------------------------------------------------------------
# the binding's refusals of device tensors
# ---------------------------------------------------------------------------

def zeros(*shape, dtype=I32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def refused(fn, good, changes):
    fn(**good())
    torch.cuda.synchronize()
    for change in changes:
        with pytest.raises((TypeError, ValueError)):
            fn(**dict(good(), **change))
    assert status() == 0


def test_binding_refuses_wrong_device_tensors():
    def plan():
        return dict(past=zeros(3), new=zeros(3), tables=zeros(3, 4), free=zeros(2), page_size=4, num_pages=64,
                    cu_seqlens=zeros(4), token_slots=zeros(5, dtype=I64), positions=zeros(5), lens=zeros(3),
                    seq_start=zeros(3, dtype=U8), free_out=zeros(2))
    refused(eng.engram_block_plan, plan, [
        dict(past=zeros(3, dtype=I64)), dict(past=zeros(6)[::2]), dict(new=zeros(2)), dict(new=zeros(3).cpu()),
        dict(tables=zeros(2, 4)), dict(tables=zeros(4, 3).t()), dict(tables=zeros(1, 4).expand(3, 4)), dict(tables=zeros(12)),
        dict(free=zeros(1)), dict(free=None, num_pages=1 << 31), dict(free_out=zeros(1)), dict(cu_seqlens=zeros(3)),
        dict(token_slots=zeros(5)), dict(positions=zeros(4)), dict(lens=zeros(2)), dict(seq_start=zeros(3)),
        dict(num_pages=-1), dict(page_size=1 << 33), dict(page_size=1.5), dict(past=None), dict(past=[1, 2, 3])])

    def release():
        return dict(tables=zeros(3, 4), lens=zeros(3), flags=zeros(3, dtype=U8), free=zeros(2), page_size=4, num_pages=64)
    refused(eng.engram_block_release, release, [
        dict(tables=zeros(4, 4)), dict(lens=zeros(2)), dict(flags=zeros(3)), dict(flags=zeros(2, dtype=U8)), dict(free=zeros(1)),
        dict(num_pages=1 << 40)])

    def select():
        work = eng.engram_beam_select_workspace(2, 3, 50, 4)
        return dict(logits=zeros(6, 50, dtype=torch.float32), scores=zeros(2, 3, dtype=torch.float32), tokens=zeros(2, 4),
                    parents=zeros(2, 4), out_scores=zeros(2, 4, dtype=torch.float32), done=zeros(2, 3, dtype=U8), end_token=1,
                    done_out=zeros(2, 4, dtype=U8), workspace=zeros(work, dtype=U8))
    refused(eng.engram_beam_select, select, [
        dict(logits=zeros(6, 50, dtype=torch.float16)), dict(logits=zeros(5, 50, dtype=torch.float32)),
        dict(logits=zeros(1, 50, dtype=torch.float32).expand(6, 50)), dict(logits=zeros(50, 6, dtype=torch.float32).t()),
        dict(logits=zeros(2, 3, 50, dtype=torch.float32)), dict(scores=zeros(6, dtype=torch.float32)), dict(scores=zeros(2, 3)),
        dict(tokens=zeros(2, 4, dtype=I64)), dict(parents=zeros(2, 3)), dict(out_scores=zeros(2, 4)), dict(tokens=zeros(1, 4)),
        dict(done=zeros(2, 4, dtype=U8)), dict(done_out=zeros(2, 3, dtype=U8)), dict(end_token=1 << 31), dict(end_token=-2),
        dict(scores=zeros(2, 6, dtype=torch.float32)[:, ::2])])
    with pytest.raises(eng.EngramError):
        eng.engram_beam_select(**dict(select(), workspace=zeros(8, dtype=U8)))

    def reorder():
        return dict(parents=zeros(2, 3), slots=zeros(2, 3), slot_src=zeros(2, 3), slot_dst=zeros(2, 3), tables=zeros(6, 4),
                    tables_out=zeros(6, 4), lens=zeros(6), page_size=4, num_pages=64, free=zeros(2), page_src=zeros(2, 3),
                    page_dst=zeros(2, 3))
    refused(eng.engram_beam_reorder, reorder, [
        dict(parents=zeros(6)), dict(slots=zeros(5)), dict(slot_src=zeros(2, 3, dtype=I64)), dict(tables=zeros(5, 4)),
        dict(tables_out=zeros(6, 5)), dict(tables_out=zeros(6, 8)[:, :4]), dict(lens=None), dict(page_size=None),
        dict(num_pages=None), dict(free=zeros(1)), dict(page_dst=zeros(5)), dict(tables=None), dict(lens=zeros(5))])

    def copy():
        return dict(state=zeros(4, 5), src=zeros(2) - 1, dst=zeros(2) - 1)
    refused(eng.engram_state_copy, copy, [
        dict(state=zeros(5)), dict(state=zeros(2, 2, 2, 2)), dict(state=zeros(5, 4).t()), dict(state=zeros(1, 5).expand(4, 5)),
        dict(src=zeros(3)), dict(dst=zeros(2, dtype=I64)), dict(src=zeros(2).cpu()), dict(state=zeros(4, 5).cpu())])
