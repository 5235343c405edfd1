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
