"""Plans of one-token rows whose slots have so much padding that the tokens take a launch of their own
(a graph captured for far more), next to those that just do not."""
import numpy as np
import pytest

from test_gpu_serve_ops import blocks_of, plan_reference, random_rows, run_plan, status

pytestmark = pytest.mark.gpu

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")


@pytest.mark.parametrize("how", ["in_place", "apart", "alias"])
@pytest.mark.parametrize("over", [0, 1, 300, 100_000])
@pytest.mark.parametrize("R", [1, 257, 1024, 1025, 3000, 4097, 8192])
def test_padded_decode(R, over, how):
    P, blocks = 16, 4
    rng = np.random.default_rng(R + over)
    new = (rng.random(R) < 0.9).astype(np.int64)
    past = rng.integers(0, blocks * P, R)
    past[rng.random(R) < 0.1] = 0
    need = sum(blocks_of(p + n, P) - blocks_of(p, P) for p, n in zip(past, new))
    tables, free, num_pages = random_rows(rng, R, blocks, P, past, need + 50)
    T = max(4096, R + 1024) + over  # the last that one launch takes, and more
    want = plan_reference(past.tolist(), new.tolist(), tables, free, P, T)
    got = run_plan(past, new, tables, free, num_pages, P, T, apart=how == "apart", alias=how == "alias")
    assert status() == 0
    for name, g, w in zip(("cu", "start", "lens", "positions", "slots", "tables", "free"), got, want):
        assert np.array_equal(g, np.asarray(w)), name
