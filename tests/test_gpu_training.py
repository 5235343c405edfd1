"""SiteTraining: a whole training step of an Engram site (lookup, 8-bit projection, gate, and their
gradients) against the same step in 64 bits on the codes that the step itself quantised, and a
few steps of gradient descent."""
import math

import pytest
import torch


pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def eng():
    if not torch.cuda.is_available():
        pytest.skip("no GPU visible")
    import hashed_gram_memory_tid2eid_amd as e
    return e


def make(eng, *, per_site, T=150, hidden=256, row_dim=96, heads=2, sites=1, scales="f32", mode="sparse", seed=0):
    L = eng.engram_layout_create(
        vocab_size=1000, compressed_vocab=600, pad_token_id=999, heads_per_order=heads, rows=[3000] * 3 if not per_site
        else [9000, 0, 0], row_dim=row_dim, table_dtype=eng.ENGRAM_DTYPE_BF16, row_pitch_bytes=2 * row_dim,
        num_sites=sites, table_split=eng.ENGRAM_TABLE_PER_SITE if per_site else eng.ENGRAM_TABLES_PER_ORDER,
        hash_floor=101)
    info = L.info
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    n_tables = 1 if per_site else 3
    tables = [torch.randn((info.rows[n], row_dim), generator=g, device=DEV) for n in range(n_tables)]
    w = torch.zeros((hidden, 3 * heads, info.seg_pitch), device=DEV)
    w[:, :, :row_dim] = torch.randn((hidden, 3 * heads, row_dim), generator=g, device=DEV) * 0.05
    w = w.flatten(1)
    site = eng.SiteTraining(L, tables, w, max_tokens=T, embed_scale=0.5, scales=scales, grad_mode=mode)
    tid2eid = (torch.arange(1000, device=DEV) % 600).int()
    tokens = torch.randint(0, 1000, (T,), generator=g, device=DEV, dtype=torch.int32)
    cu = torch.tensor([0, T // 3, T], dtype=torch.int32, device=DEV)
    row_ids = torch.empty((T, sites, 3, heads), dtype=torch.int32, device=DEV)
    eng.engram_compress_hash(L, tid2eid, tokens, cu, torch.empty(T, dtype=torch.int32, device=DEV), row_ids)
    x = torch.randn((T, 4, hidden), generator=g, device=DEV).to(BF16)
    dy = (torch.randn((T, 4, hidden), generator=g, device=DEV) * 0.1).to(BF16)
    keep = (torch.rand(T, generator=g, device=DEV) > 0.2).to(torch.uint8)
    return L, tables, w, site, row_ids, x, dy, keep


def values(q, s, n, block=1):
    s = s.double() if s.dtype == F32 else torch.exp2(s.double() - 127)
    r = torch.arange(q.shape[0], device=DEV) // block
    return (q.view(torch.float8_e4m3fn).double().view(q.shape[0], -1, 128) * s.t()[r][:, :, None]).flatten(1)[:, :n]


def close(got, want, rel):
    return float((got.double() - want).norm()) <= rel * float(want.norm())


@pytest.mark.parametrize("per_site, sites, scales, mode", [
    (False, 1, "f32", "sparse"), (True, 2, "e8m0", "sparse"), (True, 1, "f32", "accumulate"),
    (False, 2, "e8m0", "accumulate")])
@pytest.mark.parametrize("T", [1, 150])
def test_step_against_64_bits(eng, per_site, sites, scales, mode, T):
    L, tables, w, site, row_ids, x, dy, keep = make(eng, per_site=per_site, sites=sites, scales=scales, mode=mode, T=T)
    info, h, K = L.info, w.shape[0], w.shape[1]
    s = sites - 1
    y = x.clone()
    site.forward(row_ids, y, site=s, keep=keep)
    d = dy.clone()
    site.backward(d)
    torch.cuda.synchronize()
    assert eng.engram_get_error() == 0
    # forward: rows exact, the projection on the quantised operands, the gate
    cols = row_ids[:, s].reshape(T, 3 * info.heads).long()
    per = site.table_cols
    rows = torch.zeros((T, 3 * info.heads, info.seg_pitch), dtype=torch.float64, device=DEV)
    for c in range(3 * info.heads):
        rows[:, c, :info.row_dim] = (tables[c // per].double() * 0.5)[cols[:, c]]
    rows = rows.flatten(1)
    assert torch.equal(site.rows[:T], rows.float().to(BF16))
    kb, hb, tb = (-(-n // 128) for n in (K, h, T))
    rq = values(site.rows_q[:T], site.rows_s[:kb * T].view(kb, T), K)
    rt = values(site.rows_t[:, :128 * tb], site.rows_ts[:tb * K].view(tb, K), T)
    wq = values(site.w_q, site.w_s, K, 128)
    # a code is off by half a step, 2^-4 of its value, or of the smallest normal
    assert close(rq, rows, 2.0 ** -4) and close(rt, rows.t(), 2.0 ** -4) and close(wq, w.double(), 2.0 ** -4)
    v = rq @ wq.t()
    assert close(site.v[:T], v, 1e-5)
    k = keep.double()[:, None, None]
    X, V, DY = x.double(), site.v[:T].double()[:, None], dy.double()
    g = torch.sigmoid((X * V).sum(2, keepdim=True) / math.sqrt(h))
    assert close(y, X + k * g * V, 2.0 ** -8)
    # backward
    e = k * (DY * V).sum(2, keepdim=True) * g * (1 - g) / math.sqrt(h)
    assert close(d, DY + e * V, 2.0 ** -8)
    dv = (k * g * DY + e * X).sum(1)
    assert close(site.dv[:T], dv, 1e-5)
    dvq = values(site.dv_q[:T], site.dv_s[:hb * T].view(hb, T), h)
    dvt = values(site.dv_t[:, :128 * tb], site.dv_ts[:tb * h].view(tb, h), T)
    assert close(dvq, dv, 2.0 ** -4) and close(dvt, dv.t(), 2.0 ** -4)
    assert close(site.d_rows[:T], dvq @ wq, 2.0 ** -8)
    assert close(site.d_weight, dvt @ rt.t(), 1e-5)
    dr = site.d_rows[:T].double().view(T, 3 * info.heads, info.seg_pitch)[:, :, :info.row_dim] * 0.5
    for n, table in enumerate(tables):
        want = torch.zeros(table.shape, dtype=torch.float64, device=DEV)
        want.index_add_(0, cols[:, n * per:(n + 1) * per].reshape(-1), dr[:, n * per:(n + 1) * per].reshape(-1, info.row_dim))
        if mode == "sparse":
            c = int(site.count[n])
            got = torch.zeros(table.shape, dtype=F32, device=DEV)
            got[site.unique[n][:c].long()] = site.table_grads[n][:c]
        else:
            got = site.table_grads[n]
        assert close(got, want, 1e-5)


def test_smaller_call_after_a_larger_one(eng):
    """Buffers of an earlier, larger call leave no trace in a smaller one."""
    L, tables, w, site, row_ids, x, dy, keep = make(eng, per_site=True, T=150)
    fresh = eng.SiteTraining(L, tables, w, max_tokens=150, embed_scale=0.5)
    site.forward(row_ids, x.clone())
    site.backward(dy.clone())
    got = []
    for s in (site, fresh):
        y, d = x[:37].clone(), dy[:37].clone()
        s.forward(row_ids[:37], y)
        s.backward(d)
        c = int(s.count[0])
        got.append((y, d, s.d_weight.clone(), s.table_grads[0][:c].clone(), s.unique[0][:c].clone()))
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_descent_lowers_the_loss(eng):
    """Plain gradient descent on tables and weight against a fixed target of the streams."""
    L, tables, w, site, row_ids, x, _, _ = make(eng, per_site=False, T=150)
    target = x.float() + torch.randn(x.shape, generator=torch.Generator(device=DEV).manual_seed(9), device=DEV) * 0.2
    losses = []
    for _ in range(6):
        y = x.clone()
        site.forward(row_ids, y)
        diff = y.float() - target
        losses.append(float((diff * diff).sum()))
        d = diff.to(BF16)
        site.backward(d)
        w -= 2e-4 * site.d_weight
        site.load_weight(w)
        for t, g, u, c in zip(tables, site.table_grads, site.unique, site.count):
            c = int(c)
            t[u[:c].long()] -= 0.05 * g[:c]
    assert all(b < a for a, b in zip(losses, losses[1:])), losses


def test_refusals(eng):
    L, tables, w, site, row_ids, x, dy, keep = make(eng, per_site=True, T=20)
    with pytest.raises(RuntimeError):
        site.backward(dy)
    with pytest.raises(ValueError):
        site.forward(row_ids, torch.cat([x, x]))
    with pytest.raises(ValueError):
        site.forward(row_ids, x, site=1)
    with pytest.raises(ValueError):
        eng.SiteTraining(L, tables * 2, w, max_tokens=20)
    with pytest.raises(ValueError):
        eng.SiteTraining(L, tables, w[:, :64], max_tokens=20)
    with pytest.raises(ValueError):
        eng.SiteTraining(L, tables, w, max_tokens=20, scales="int8")
    site.forward(row_ids, x.clone())
    with pytest.raises(ValueError):
        site.backward(dy[:3])
