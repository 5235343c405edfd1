"""Sizes past 32 bits are refused by the serving operators' binding: ctypes would cut them down to
their low 32 bits without a word.  (Tensors without elements, so that none of it needs memory.)"""
import pytest
import torch

pytestmark = pytest.mark.gpu

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")
I32, U8, F32 = torch.int32, torch.uint8, torch.float32


def empty(*shape, dtype=I32):
    return torch.zeros(shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("shape", [(1 << 31, 0), ((1 << 32) + 3, 0), (0, 1 << 31), (0, (1 << 32) + 3)])
def test_a_matrix_is_refused(shape):
    from hashed_gram_memory_tid2eid_amd import _tensor_args as ta
    with pytest.raises(ValueError):
        ta.matrix(empty(*shape), "x", I32, torch.cuda.current_device())
    assert ta.matrix(empty(0, (1 << 31) - 1), "x", I32, torch.cuda.current_device())[1:3] == (0, (1 << 31) - 1)


def test_tables_are_refused():
    wide = empty(0, (1 << 32) + 3)
    with pytest.raises(ValueError):
        eng.engram_block_plan(empty(0), empty(0), wide, empty(2), page_size=4, num_pages=64, cu_seqlens=empty(1),
                              token_slots=empty(0, dtype=torch.int64))
    with pytest.raises(ValueError):
        eng.engram_block_release(wide, empty(0), empty(0, dtype=U8), empty(2), page_size=4, num_pages=64)
    with pytest.raises(ValueError):
        eng.engram_beam_reorder(empty(0, 4), tables=wide, lens=empty(0), page_size=4, num_pages=64)


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 4])
def test_a_selection_is_refused(n):
    work = empty(64, dtype=U8)
    with pytest.raises(ValueError):
        eng.engram_beam_select(empty(0, 10, dtype=F32), empty(0, 4, dtype=F32), empty(0, n), empty(0, n), empty(0, n, dtype=F32),
                               workspace=work)
