"""The lookup gradient with every length of chunk (8, 16 and 32 places; short lists have 4): more
columns or more places than the other tests', so that runs go on over several steps of a chunk, end
anywhere inside one, and cross chunks and units of 32 chunks.  Whole numbers: every sum is exact in any
order, and a bf16 gradient is that sum rounded once."""
import pytest
import torch

from test_gpu_train_ops import BF16, DEV, F32, eng, gen, grad_ref, no_device_error, run_grad  # noqa: F401

pytestmark = pytest.mark.gpu
ROWS = 4000


def sorted_ids(kind, n):
    i = torch.arange(n, device=DEV)
    if kind == "one":
        return torch.full((n,), 17, device=DEV)
    if kind == "runs":  # 1, 2, 3, ... places
        return torch.sqrt(2.0 * i.double()).long() % ROWS
    if kind == "growing":  # 1, 3, 9, ... places
        return (torch.log(2.0 * i.double() + 1) / 1.0986122886681098).long()
    if kind == "even":  # every run whole chunks, of any length of chunk
        return i // 64 % ROWS
    if kind == "none":
        return torch.full((n,), -1, device=DEV)
    if kind == "half":  # the places of rows end inside a chunk, the others have none
        return torch.where(i < n // 2 + 3, i // 45, -1)
    assert kind == "last"
    return torch.where(i == n - 1, ROWS - 1, -1)


# the chunk's length is in front; 131,072 lanes of 8 columns each have to be left
CLASSES = [(8, 2101, 4096), (16, 4203, 4096), (32, 8505, 4096), (32, 8477, 4093), (8, 33_003, 256), (16, 65_541, 256),
           (32, 132_107, 256), (32, 264_211, 122)]


@pytest.mark.parametrize("chunk, n, dim", CLASSES)
@pytest.mark.parametrize("kind", ["one", "runs", "growing", "even", "none", "half", "last"])
def test_runs_over_longer_chunks(eng, chunk, n, dim, kind):
    lanes = n * next(g for g in (128, 256, 4096) if g >= dim) // 8
    assert chunk * 131072 <= lanes and (chunk == 32 or lanes < 2 * chunk * 131072) and n % chunk
    g = gen(n + dim)
    ids = sorted_ids(kind, n)[torch.randperm(n, generator=g, device=DEV)].int().view(n, 1)
    dout = torch.randint(-4, 5, (n, dim), generator=g, device=DEV).to(BF16)
    ref, _, terms = grad_ref(ids, dout, ROWS, dim, dim, 2.0)
    named = terms > 0
    assert torch.equal(run_grad(eng, ids, dout, ROWS, dim, dim, 2.0, "dense", F32).double(), ref)
    assert torch.equal(run_grad(eng, ids, dout.float(), ROWS, dim, dim, 2.0, "dense", BF16), ref.float().to(BF16))
    grad, unique, count = run_grad(eng, ids, dout, ROWS, dim, dim, 2.0, "sparse", F32)
    assert count == int(named.sum())
    assert torch.equal(unique[:count].long(), torch.nonzero(named).flatten()) and bool((unique[count:] == -1).all())
    assert torch.equal(grad[:count].double(), ref[named]) and bool((grad[count:] == 3.0).all())
    start = torch.randint(-9, 10, (ROWS, dim), generator=g, device=DEV).float()
    added = run_grad(eng, ids, dout, ROWS, dim, dim, 2.0, "accumulate", F32, start)
    assert torch.equal(added.double(), ref + start.double())


@pytest.mark.parametrize("T, cols, dim, seg", [(5501, 24, 250, 256), (1403, 24, 256, 256), (8501, 3, 1000, 1024)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_columns_of_ids_over_longer_chunks(eng, T, cols, dim, seg, dtype):
    """Several places a token, segments with padding, ids that repeat at random."""
    g = gen(T)
    ids = torch.randint(-1, 997, (T, cols), generator=g, device=DEV, dtype=torch.int32)
    ids[torch.rand((T, cols), generator=g, device=DEV) < 0.2] = 500
    dout = torch.randint(-4, 5, (T, cols * seg), generator=g, device=DEV).to(dtype)
    ref, _, terms = grad_ref(ids, dout, 997, dim, seg, 1.0)
    assert torch.equal(run_grad(eng, ids, dout, 997, dim, seg, 1.0, "dense", F32).double(), ref)
    grad, unique, count = run_grad(eng, ids, dout, 997, dim, seg, 1.0, "sparse", F32)
    assert torch.equal(unique[:count].long(), torch.nonzero(terms).flatten())
    assert torch.equal(grad[:count].double(), ref[terms > 0])
