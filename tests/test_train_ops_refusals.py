"""Refusals of the training operators, on the host: every call below is turned down by its
argument checks before anything is launched, so no GPU is needed.  The C entry points get
made-up aligned addresses that nothing dereferences."""
import ctypes

import pytest
import torch

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")
lib = eng._lib
P = 1 << 20  # a 256-byte aligned address
BF16, F32 = eng.ENGRAM_DTYPE_BF16, eng.ENGRAM_DTYPE_F32


def call(fn, base, **change):
    args = dict(base, **change)
    assert set(change) <= set(base)
    return fn(*args.values())


EMBED = dict(table=P, table_dtype=BF16, rows=100, dim=64, table_ld=64, ids=P, T=4, cols=3, ids_ld=3, scale=1.0, out=P,
             out_dtype=BF16, out_ld=192, seg=64, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(table=None), "ARG"), (dict(ids=None), "ARG"), (dict(out=None), "ARG"), (dict(table_dtype=1), "ARG"),
    (dict(out_dtype=0), "ARG"), (dict(rows=0), "ARG"), (dict(rows=1 << 31), "ARG"), (dict(dim=0), "ARG"),
    (dict(table_ld=63), "ARG"), (dict(T=-1), "ARG"), (dict(cols=0), "ARG"), (dict(ids_ld=2), "ARG"),
    (dict(seg=63), "ARG"), (dict(out_ld=191), "ARG"), (dict(scale=float("inf")), "ARG"),
    (dict(scale=float("nan")), "ARG"), (dict(table=P + 1), "ALIGN"), (dict(out=P + 1), "ALIGN"), (dict(ids=P + 2), "ALIGN"),
    (dict(seg=1 << 30, out_ld=3 << 30), "UNSUPPORTED"), (dict(T=1 << 31), "UNSUPPORTED"),
])
def test_embed_refuses(change, status):
    assert call(lib.engram_embed, EMBED, **change) == eng.STATUS["ENGRAM_E_" + status]


def test_embed_of_no_tokens_is_nothing():
    assert call(lib.engram_embed, EMBED, T=0, ids=None, out=None, table=None) == 0


GRAD = dict(ids=P, T=4, cols=3, ids_ld=3, rows=100, dim=64, scale=1.0, dout=P, dout_dtype=BF16, dout_ld=192, seg=64, mode=2,
            grad=P, grad_dtype=F32, grad_ld=64, unique=P, count=P, work=P, work_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(ids=None), "ARG"), (dict(dout=None), "ARG"), (dict(grad=None), "ARG"), (dict(unique=None), "ARG"),
    (dict(count=None), "ARG"), (dict(work=None), "ARG"), (dict(mode=3), "ARG"), (dict(mode=-1), "ARG"),
    (dict(dout_dtype=1), "ARG"), (dict(grad_dtype=1), "ARG"), (dict(grad_ld=63), "ARG"), (dict(dout_ld=191), "ARG"),
    (dict(scale=float("nan")), "ARG"), (dict(rows=0), "ARG"), (dict(work_bytes=0), "SCRATCH"), (dict(work=P + 16), "ALIGN"),
    (dict(grad=P + 2), "ALIGN"), (dict(dout=P + 1), "ALIGN"), (dict(count=P + 1), "ALIGN"),
    (dict(T=1 << 30), "UNSUPPORTED"),
])
def test_embed_grad_refuses(change, status):
    assert call(lib.engram_embed_grad, GRAD, **change) == eng.STATUS["ENGRAM_E_" + status]


def test_embed_grad_workspace():
    assert eng.engram_embed_grad_workspace(0, 10, 8) >= 0
    small, large = (eng.engram_embed_grad_workspace(n, 1000, 64) for n in (1000, 100_000))
    assert 0 < small < large
    # exactly what the workspace function says is enough; a byte less is not
    assert call(lib.engram_embed_grad, GRAD, work_bytes=eng.engram_embed_grad_workspace(12, 100, 64) - 1) == \
        eng.ENGRAM_E_SCRATCH
    for args in ((-1, 10, 8), (10, 0, 8), (10, 10, 0)):
        with pytest.raises(eng.EngramError):
            eng.engram_embed_grad_workspace(*args)
    with pytest.raises(eng.EngramError):
        eng.engram_embed_grad_workspace((1 << 30) + 1, 10, 8)
    n = ctypes.c_int64()
    assert lib.engram_embed_grad_workspace(10, 10, 8, None) == eng.ENGRAM_E_ARG
    assert lib.engram_embed_grad_workspace(10, 10, 8, ctypes.byref(n)) == 0


QUANT = dict(x=P, x_dtype=BF16, M=100, K=200, ld=200, kind=0, block=1, q=P, q_ld=256, s=P, qt=P, qt_ld=128, st=P, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(x=None), "ARG"), (dict(x_dtype=1), "ARG"), (dict(M=-1), "ARG"), (dict(K=-1), "ARG"), (dict(ld=199), "ARG"),
    (dict(kind=2), "ARG"), (dict(block=64), "ARG"), (dict(q=None, qt=None), "ARG"), (dict(s=None), "ARG"),
    (dict(st=None), "ARG"), (dict(q_ld=255), "ALIGN"), (dict(q_ld=240), "ALIGN"), (dict(q_ld=264), "ALIGN"),
    (dict(qt_ld=112), "ALIGN"), (dict(q=P + 8), "ALIGN"), (dict(qt=P + 8), "ALIGN"), (dict(s=P + 1), "ALIGN"),
    (dict(st=P + 2), "ALIGN"), (dict(x=P + 1), "ALIGN"),
    (dict(M=(1 << 31) - 1, qt=None, st=None), "UNSUPPORTED"),
    (dict(M=1 << 30, K=1 << 14, ld=1 << 14, q_ld=1 << 14, qt=None, st=None), "UNSUPPORTED"),
])
def test_quantize_refuses(change, status):
    assert call(lib.engram_fp8_quantize, QUANT, **change) == eng.STATUS["ENGRAM_E_" + status]


def test_quantize_of_nothing_is_nothing():
    assert call(lib.engram_fp8_quantize, QUANT, M=0, x=None) == 0
    assert call(lib.engram_fp8_quantize, QUANT, K=0, x=None) == 0


MATMUL = dict(a=P, a_ld=256, sa=P, b=P, b_ld=256, sb=P, block=128, kind=0, M=64, N=96, K=256, c=P, c_dtype=F32, c_ld=96,
              work=P, work_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(a=None), "ARG"), (dict(sa=None), "ARG"), (dict(b=None), "ARG"), (dict(sb=None), "ARG"), (dict(c=None), "ARG"),
    (dict(block=2), "ARG"), (dict(kind=2), "ARG"), (dict(c_dtype=1), "ARG"), (dict(M=-1), "ARG"), (dict(N=-1), "ARG"),
    (dict(K=0), "ARG"), (dict(K=200), "ARG"), (dict(a_ld=128), "ARG"), (dict(b_ld=128), "ARG"), (dict(c_ld=95), "ARG"),
    (dict(a_ld=264), "ALIGN"), (dict(b_ld=264), "ALIGN"), (dict(a=P + 8), "ALIGN"), (dict(b=P + 8), "ALIGN"),
    (dict(sa=P + 2), "ALIGN"), (dict(c=P + 2), "ALIGN"), (dict(a_ld=1 << 23), "UNSUPPORTED"),
    (dict(M=(1 << 31) - 1), "UNSUPPORTED"),
])
def test_matmul_refuses(change, status):
    assert call(lib.engram_fp8_matmul, MATMUL, **change) == eng.STATUS["ENGRAM_E_" + status]


def test_matmul_workspace():
    need = eng.engram_fp8_matmul_workspace(200, 4096, 6144)
    assert need > 0  # too few tiles for the chip: K is split
    assert call(lib.engram_fp8_matmul, MATMUL, M=200, N=4096, K=6144, a_ld=6144, b_ld=6144, c_ld=4096, work_bytes=need - 1) \
        == eng.ENGRAM_E_SCRATCH
    assert call(lib.engram_fp8_matmul, MATMUL, M=200, N=4096, K=6144, a_ld=6144, b_ld=6144, c_ld=4096, work=None) == \
        eng.ENGRAM_E_SCRATCH
    assert eng.engram_fp8_matmul_workspace(65_536, 4096, 6144) == 0
    assert eng.engram_fp8_matmul_workspace(16, 4096, 6144) == 0  # a few rows need none
    assert eng.engram_fp8_matmul_workspace(0, 4096, 6144) == 0
    assert eng.engram_fp8_matmul_workspace(5, 7, 100) == eng.engram_fp8_matmul_workspace(5, 7, 128)
    with pytest.raises(eng.EngramError):
        eng.engram_fp8_matmul_workspace(-1, 4096, 6144)


GATE = dict(v=P, x=P, keep=None, dy=P, hidden=64, hc=4, dx=P, dv=P, T=3, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(v=None), "ARG"), (dict(x=None), "ARG"), (dict(dy=None), "ARG"), (dict(dx=None), "ARG"), (dict(dv=None), "ARG"),
    (dict(T=-1), "ARG"), (dict(hc=2), "UNSUPPORTED"), (dict(hidden=8200), "UNSUPPORTED"), (dict(hidden=60), "ALIGN"),
    (dict(hidden=0), "ALIGN"), (dict(v=P + 4), "ALIGN"), (dict(dx=P + 8), "ALIGN"), (dict(dv=P + 4), "ALIGN"),
])
def test_gate_backward_refuses(change, status):
    assert call(lib.engram_gate_add_backward, GATE, **change) == eng.STATUS["ENGRAM_E_" + status]


def test_gate_backward_of_no_tokens_is_nothing():
    assert call(lib.engram_gate_add_backward, GATE, T=0, v=None) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    ids, table, out = torch.zeros(4, dtype=torch.int32), torch.zeros(8, 16), torch.zeros(4, 16)
    with pytest.raises(TypeError):
        eng.engram_embed(table, ids, out)  # host memory
    with pytest.raises(TypeError):
        eng.engram_embed(table.half(), ids, out)
    with pytest.raises(ValueError):
        eng.engram_embed_grad(ids, out, table, rows=8, mode="sum")
    with pytest.raises(ValueError):
        eng.engram_fp8_quantize(torch.zeros(4, 128), None, None, block_rows=2)
