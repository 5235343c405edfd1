"""Refusals of the serving operators, on the host: every call below is turned down by its
argument checks before anything is launched, so no GPU is needed.  The C entry points get
made-up aligned addresses that nothing dereferences."""
import ctypes

import pytest
import torch

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")
lib = eng._lib
P = 1 << 20  # an aligned address
BF16, F32 = eng.ENGRAM_DTYPE_BF16, eng.ENGRAM_DTYPE_F32


def call(fn, base, **change):
    assert set(change) <= set(base)
    return fn(*dict(base, **change).values())


PLAN = dict(past=P, new=P, R=4, page_size=16, tables=P, ld=8, blocks=8, free=P, free_out=P, pages=100, cu=P, start=P, lens=P,
            T=10, positions=P, slots=P, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(past=None), "ARG"), (dict(new=None), "ARG"), (dict(tables=None), "ARG"), (dict(free=None), "ARG"),
    (dict(free_out=None), "ARG"), (dict(cu=None), "ARG"), (dict(slots=None), "ARG"), (dict(R=-1), "ARG"),
    (dict(page_size=0), "ARG"), (dict(ld=7), "ARG"), (dict(blocks=-1), "ARG"), (dict(pages=-1), "ARG"), (dict(T=-1), "ARG"),
    (dict(R=8193), "UNSUPPORTED"), (dict(pages=1 << 30), "UNSUPPORTED"), (dict(T=(1 << 31) - 1), "UNSUPPORTED"),
    (dict(page_size=1 << 28), "UNSUPPORTED"), (dict(past=P + 1), "ALIGN"), (dict(new=P + 2), "ALIGN"),
    (dict(tables=P + 2), "ALIGN"), (dict(free=P + 1), "ALIGN"), (dict(free_out=P + 1), "ALIGN"), (dict(cu=P + 1), "ALIGN"),
    (dict(lens=P + 2), "ALIGN"), (dict(positions=P + 1), "ALIGN"), (dict(slots=P + 4), "ALIGN"),
])
def test_plan_refuses(change, status):
    assert call(lib.engram_block_plan, PLAN, **change) == eng.STATUS["ENGRAM_E_" + status]


RELEASE = dict(tables=P, ld=8, blocks=8, lens=P, flags=P, R=4, page_size=16, free=P, pages=100, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(tables=None), "ARG"), (dict(lens=None), "ARG"), (dict(flags=None), "ARG"), (dict(free=None), "ARG"),
    (dict(R=-1), "ARG"), (dict(page_size=0), "ARG"), (dict(ld=7), "ARG"), (dict(pages=-1), "ARG"),
    (dict(R=1 << 24), "UNSUPPORTED"), (dict(page_size=1 << 28), "UNSUPPORTED"), (dict(tables=P + 1), "ALIGN"),
    (dict(lens=P + 1), "ALIGN"), (dict(free=P + 2), "ALIGN"),
])
def test_release_refuses(change, status):
    assert call(lib.engram_block_release, RELEASE, **change) == eng.STATUS["ENGRAM_E_" + status]


SELECT = dict(logits=P, dtype=BF16, ld=1000, G=3, K=4, V=1000, scores=P, done=P, end=7, n=8, tokens=P, parents=P, out=P,
              out_done=P, work=P, work_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(logits=None), "ARG"), (dict(scores=None), "ARG"), (dict(tokens=None), "ARG"), (dict(parents=None), "ARG"),
    (dict(out=None), "ARG"), (dict(work=None), "ARG"), (dict(dtype=1), "ARG"), (dict(ld=999), "ARG"), (dict(G=-1), "ARG"),
    (dict(K=0), "ARG"), (dict(V=0), "ARG"), (dict(n=0), "ARG"), (dict(end=-2), "ARG"), (dict(end=1000), "ARG"),
    (dict(end=-1), "ARG"), (dict(K=65), "UNSUPPORTED"), (dict(n=65), "UNSUPPORTED"),
    (dict(V=(1 << 24) + 1, ld=1 << 25), "UNSUPPORTED"), (dict(G=1 << 19), "UNSUPPORTED"),
    (dict(G=1 << 15, V=1 << 24, ld=1 << 24), "UNSUPPORTED"), (dict(work_bytes=0), "SCRATCH"), (dict(logits=P + 1), "ALIGN"),
    (dict(logits=P + 2, dtype=F32), "ALIGN"), (dict(scores=P + 1), "ALIGN"), (dict(tokens=P + 1), "ALIGN"),
    (dict(parents=P + 1), "ALIGN"), (dict(out=P + 1), "ALIGN"), (dict(work=P + 8), "ALIGN"),
])
def test_select_refuses(change, status):
    assert call(lib.engram_beam_select, SELECT, **change) == eng.STATUS["ENGRAM_E_" + status]


def test_select_workspace():
    need = eng.engram_beam_select_workspace(3, 4, 1000, 8)
    assert call(lib.engram_beam_select, SELECT, work_bytes=need - 1) == eng.ENGRAM_E_SCRATCH
    # a workspace for G requests serves every smaller call
    for K, V in ((1, 129_280), (4, 129_280), (8, 1000), (64, 32_001)):
        sizes = [eng.engram_beam_select_workspace(G, K, V, 8) for G in range(0, 600, 7)]
        assert sizes == sorted(sizes)
    n = ctypes.c_int64()
    assert lib.engram_beam_select_workspace(1, 1, 1, 1, None) == eng.ENGRAM_E_ARG
    for args in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 1, 0, 1), (1, 1, 1, 0)):
        assert lib.engram_beam_select_workspace(*args, ctypes.byref(n)) == eng.ENGRAM_E_ARG
    with pytest.raises(ValueError):
        eng.engram_beam_select_workspace(1 << 32, 1, 1, 1)


REORDER = dict(parents=P, G=3, K=4, store=None, slots=P, slots_out=P, slot_src=P, slot_dst=P, tables=P, tables_out=P, ld=8,
               blocks=8, lens=P, page_size=16, free=P, pages=100, page_src=P, page_dst=P, stream=None)
NO_TABLES = dict(tables=None, tables_out=None, free=None, page_src=None, page_dst=None)
NO_SLOTS = dict(slots=None, slots_out=None, slot_src=None, slot_dst=None)


@pytest.mark.parametrize("change, status", [
    (dict(parents=None), "ARG"), (dict(G=-1), "ARG"), (dict(K=0), "ARG"), (dict(slots_out=None), "ARG"),
    (dict(**NO_TABLES, **NO_SLOTS), "ARG"), (dict(NO_SLOTS, slots_out=P), "ARG"), (dict(NO_SLOTS, slot_src=P), "ARG"),
    (dict(NO_SLOTS, store=P), "ARG"), (dict(tables_out=None), "ARG"), (dict(lens=None), "ARG"), (dict(page_size=0), "ARG"),
    (dict(ld=7), "ARG"), (dict(NO_TABLES, free=P), "ARG"), (dict(NO_TABLES, page_src=P), "ARG"),
    (dict(NO_TABLES, tables_out=P), "ARG"), (dict(K=65), "UNSUPPORTED"), (dict(G=1 << 20), "UNSUPPORTED"),
    (dict(page_size=1 << 28), "UNSUPPORTED"), (dict(page_size=1, ld=1 << 25, blocks=1 << 25), "UNSUPPORTED"),
    (dict(parents=P + 1), "ALIGN"), (dict(slots=P + 1), "ALIGN"), (dict(tables=P + 1), "ALIGN"), (dict(free=P + 1), "ALIGN"),
    (dict(page_dst=P + 1), "ALIGN"),
])
def test_reorder_refuses(change, status):
    assert call(lib.engram_beam_reorder, REORDER, **change) == eng.STATUS["ENGRAM_E_" + status]


COPY = dict(state=P, planes=2, plane_pitch=1 << 16, rows=16, row_pitch=4096, row_bytes=4096, src=P, dst=P, n=4, stream=None)


@pytest.mark.parametrize("change, status", [
    (dict(state=None), "ARG"), (dict(src=None), "ARG"), (dict(dst=None), "ARG"), (dict(planes=-1), "ARG"),
    (dict(plane_pitch=-1), "ARG"), (dict(rows=-1), "ARG"), (dict(row_bytes=0), "ARG"), (dict(row_pitch=4095), "ARG"),
    (dict(n=-1), "ARG"), (dict(rows=1 << 31), "UNSUPPORTED"), (dict(row_pitch=1 << 27, row_bytes=1 << 26), "UNSUPPORTED"),
    (dict(planes=1 << 23), "UNSUPPORTED"), (dict(src=P + 1), "ALIGN"), (dict(dst=P + 1), "ALIGN"),
])
def test_copy_refuses(change, status):
    assert call(lib.engram_state_copy, COPY, **change) == eng.STATUS["ENGRAM_E_" + status]


def test_calls_with_nothing_to_do_launch_nothing():
    assert call(lib.engram_block_release, RELEASE, R=0, tables=None, lens=None, flags=None) == 0
    assert call(lib.engram_beam_select, SELECT, G=0, logits=None, scores=None) == 0
    assert call(lib.engram_beam_reorder, REORDER, G=0, parents=None) == 0
    assert call(lib.engram_state_copy, COPY, n=0, src=None, dst=None) == 0
    assert call(lib.engram_state_copy, COPY, planes=0) == 0


def test_binding_refuses_what_is_not_a_device_tensor():
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    with pytest.raises((TypeError, ValueError)):
        eng.engram_block_plan(i32(2), i32(2), i32(2, 3), i32(4), page_size=4, num_pages=100, cu_seqlens=i32(3),
                              token_slots=torch.zeros(5, dtype=torch.int64))
    with pytest.raises((TypeError, ValueError)):
        eng.engram_block_release(i32(2, 3), i32(2), torch.zeros(2, dtype=torch.uint8), i32(4), page_size=4, num_pages=100)
    with pytest.raises((TypeError, ValueError)):
        eng.engram_beam_reorder(i32(2, 3), slots=i32(2, 3))
    with pytest.raises((TypeError, ValueError)):
        eng.engram_state_copy(i32(4, 4), i32(2), i32(2))
    with pytest.raises((TypeError, ValueError)):
        eng.engram_beam_select(torch.zeros(4, 10), torch.zeros(2, 2), i32(2, 2), i32(2, 2), torch.zeros(2, 2), workspace=i32(64))


def test_tensor_arguments_of_the_wrong_kind():
    from hashed_gram_memory_tid2eid_amd import _tensor_args as ta
    host = torch.zeros(4, dtype=torch.int32)
    assert ta.address(None, "x", torch.int32, 4, 0) is None
    for call in (lambda t: ta.device(t, "x"), lambda t: ta.address(t, "x", torch.int32, 1, 0),
                 lambda t: ta.matrix(t, "x", torch.int32, 0)):
        for wrong in (host, [1, 2], 7, "x"):
            with pytest.raises(TypeError):
                call(wrong)
    for args in ((), (host,), (host, "x", torch.int32, 1, 0, 0)):
        with pytest.raises(TypeError):
            ta.address(*args)
    with pytest.raises(TypeError):
        ta.device(host, 3)
    for bad in (-1, 1 << 31, 1.5):
        with pytest.raises(ValueError):
            eng.serve_ops._count(bad, "x")
    assert eng.serve_ops._count(7, "x") == 7
