"""Serving operators of batches and states without anything in them: empty tensors, whose addresses are
null, are no fault."""
import pytest
import torch

from test_gpu_serve_ops import dev, small_store, status, zeros

pytestmark = pytest.mark.gpu

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")


@pytest.mark.parametrize("with_slots", [True, False])
@pytest.mark.parametrize("with_tables", [True, False])
def test_reordering_of_no_requests(with_slots, with_tables):
    args = {}
    if with_slots:
        args.update(slots=zeros(0, 4), slot_src=zeros(0, 4), slot_dst=zeros(0, 4), store=small_store(4)[0])
    if with_tables:
        words = dev([5])
        args.update(tables=zeros(0, 8), lens=zeros(0), page_size=4, num_pages=20, free=words, page_src=zeros(0, 4),
                    page_dst=zeros(0, 4))
    if not args:
        with pytest.raises((ValueError, eng.EngramError)):  # neither slots nor tables, of as many requests as you like
            eng.engram_beam_reorder(zeros(2, 4))
        return
    eng.engram_beam_reorder(zeros(0, 4), **args)
    assert status() == 0 and (not with_tables or words.tolist() == [5])


def test_selection_of_no_requests():
    e = torch.empty((0, 4), device="cuda")
    eng.engram_beam_select(torch.empty((0, 50), device="cuda"), e, zeros(0, 4), zeros(0, 4), e.clone(),
                           workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert status() == 0


def test_release_of_no_rows():
    words = dev([5])
    eng.engram_block_release(zeros(0, 4), zeros(0), zeros(0, dtype=torch.uint8), words, page_size=4, num_pages=20)
    assert status() == 0 and words.tolist() == [5]


@pytest.mark.parametrize("shape", [(0, 8), (3, 0, 8), (0, 5, 8), (3, 5, 0)])
def test_copy_of_a_state_without_rows(shape):
    state = torch.zeros(shape, device="cuda")
    eng.engram_state_copy(state, dev([-1, 3, 0]), dev([0, -1, 0]))
    assert status() == 0
    if shape[-2] == 0 and 0 not in shape[:-2]:
        eng.engram_state_copy(state, dev([1]), dev([2]))
        assert status() == eng.ENGRAM_E_SLOT_RANGE
