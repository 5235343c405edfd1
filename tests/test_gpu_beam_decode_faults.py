"""BeamDecode after a fault: what a start or a plan that does not fit leaves behind, on states that
have served other prompts before."""
import pytest
import torch

from test_gpu_serve_ops import dev, status, unpack

pytestmark = pytest.mark.gpu

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")


def used_before(K, num_pages):
    """Two requests over pages of 4 tokens, whose tables name pages of earlier prompts."""
    d = eng.BeamDecode(None, requests=2, beams=K, max_len=20, page_size=4, vocab=10, num_pages=num_pages)
    d.start(dev([8, 4]), 12)
    d.finish()
    assert status() == 0
    return d


def all_free(d):
    return unpack(d.free.cpu(), d.num_pages).all()


@pytest.mark.parametrize("K", [1, 3])
@pytest.mark.parametrize("lens, places, code", [
    ([12, 13], 25, "PAGES"),          # seven pages of six
    ([6, 7], 12, "SEQLENS"),          # a token more than places
    ([6, -1], 30, "SEQLENS"), ([6, 21], 30, "SEQLENS"),
])
def test_start_of_prompts_that_do_not_fit_takes_nothing(K, lens, places, code):
    d = used_before(K, 6)
    d.start(dev(lens), places)
    assert status() == eng.STATUS["ENGRAM_E_" + code]
    assert d.lens.tolist() == [0] * (2 * K) and all_free(d)
    assert d.cu_seqlens.tolist() == [0] * 3 and (d.token_slots == -1).all()
    # rows that hold nothing: a token of each lies on a page of its own
    d.plan()
    assert status() == 0
    slots = d.token_slots.tolist()
    assert len(set(slots)) == 2 * K and min(slots) >= 0 and d.positions.tolist() == [0] * (2 * K)
    d.finish()
    assert status() == 0 and all_free(d)
    d.start(dev([8, 4]), 12)
    assert status() == 0 and d.lens.tolist() == [8] * K + [4] * K


@pytest.mark.parametrize("lens", [[8, 5], [9, 10], [1, 1]])
def test_start_whose_last_pages_do_not_fit(lens):
    """The first beams have their prompts, the others no page of their own; finish gives all of it back."""
    K, own = 3, sum(-(-n // 4) for n in lens)
    d = used_before(K, max(own, 5))
    d.start(dev(lens), sum(lens))
    assert status() == eng.ENGRAM_E_PAGES
    assert d.lens.view(2, K).tolist() == [[n] + [n // 4 * 4] * (K - 1) for n in lens]
    assert int(unpack(d.free.cpu(), d.num_pages).sum()) == d.num_pages - own
    d.finish()
    assert status() == 0 and all_free(d)


def test_start_that_fits_again_after_a_fault():
    d = used_before(2, 6)
    for _ in range(2):
        d.start(dev([13, 12]), 25)
        assert status() == eng.ENGRAM_E_PAGES
        d.finish()
        d.start(dev([6, 3]), 9)
        assert status() == 0 and d.lens.tolist() == [6, 6, 3, 3]
        assert int(unpack(d.free.cpu(), d.num_pages).sum()) == 6 - 5
        tables = d.tables.tolist()
        last = [tables[r][n // 4] for r, n in enumerate(d.lens.tolist())]
        assert len(set(last)) == 4 and tables[0][0] == tables[1][0]
        d.finish()
        assert status() == 0 and all_free(d)


# ---------------------------------------------------------------------------
# caches
# ---------------------------------------------------------------------------

def test_caches_that_cannot_be_copied_are_refused_when_made():
    """Not at the first selection, whose beams have moved by then."""
    size = dict(requests=2, beams=2, max_len=8, page_size=2, vocab=10)
    zeros = lambda *s: torch.zeros(s, device="cuda")  # noqa: E731
    for cache in (zeros(8), zeros(2, 2, 8, 4), zeros(4, 16).t(), zeros(1, 4).expand(16, 4), zeros(1, 16, 4).expand(2, 16, 4),
                  zeros(2, 16, 4).cpu(), zeros(40).as_strided((2, 16, 2), (1, 2, 1))):
        with pytest.raises((TypeError, ValueError)):
            eng.BeamDecode(None, caches=[zeros(16, 4), cache], **size)
    with pytest.raises(eng.EngramError):  # more planes than a copy of these beams takes
        eng.BeamDecode(None, caches=[torch.zeros((1 << 22, 16, 1), dtype=torch.uint8, device="cuda")], **size)
    d = eng.BeamDecode(None, caches=[zeros(16, 4), zeros(3, 17, 5), zeros(16, 2, 4).transpose(0, 1)], **size)
    d.start(dev([1, 1]), 2)
    d.first(torch.zeros((2, 10), device="cuda"))
    assert status() == 0


# ---------------------------------------------------------------------------
# lengths
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("max_len, P, holds", [(17, 16, 32), (16, 16, 16), (1, 1, 1), (5, 3, 6)])
def test_max_len_is_what_plan_keeps_to(max_len, P, holds):
    d = eng.BeamDecode(None, requests=2, beams=2, max_len=max_len, page_size=P, vocab=10)
    assert d.max_len == holds
    d.start(dev([holds, 1]), holds + 1)
    d.finish()
    d.start(dev([1, 1]), 2)
    d.first(torch.zeros((2, 10), device="cuda"))
    for i in range(holds - 1):
        d.plan()
        assert d.positions.tolist() == [i + 1] * 4
        d.select(torch.zeros((4, 10), device="cuda"))
    assert status() == 0
    d.plan()
    assert status() == eng.ENGRAM_E_SEQLENS and d.lens.tolist() == [holds] * 4


def test_the_loop_of_the_readme_ends():
    """As it stands there, with a request that has nothing to select from (its beams are never done)."""
    import os
    import re

    import engram_inputs as ei
    from engram_harness import DEV, Site
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "README.md")) as f:
        code = next(c for c in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "BeamDecode(" in c)
    cfg = ei.get_config("decode_tiny")
    lens = [4085, 4070, 3, 1, 77, 4085, 16, 2]
    total = sum(lens)
    logits = torch.randn((32, 129_280), device="cuda")
    logits[:, cfg.vocab:] = -torch.inf
    logits[8:12] = torch.nan
    names = dict(engram=Site(cfg, max_tokens=total).site, kv=torch.zeros((8 * 4 * 256, 16), device="cuda"),
                 prompt_lens=dev(lens), num_tokens=total, longest_prompt=max(lens),
                 prompt_tokens=torch.zeros(total, dtype=torch.int32, device="cuda"),
                 prompt_streams=ei.make_streams(cfg, total, DEV), streams=ei.make_streams(cfg, 32, DEV), logits=logits,
                 prompt_logits=logits[::4].contiguous())
    exec(code, names)
    d = names["d"]
    assert status() == 0 and all_free(d) and not d.done[2].any()


@pytest.mark.parametrize("end_token", [10, 11, -2])
def test_an_end_token_outside_the_vocabulary_is_refused_when_made(end_token):
    size = dict(requests=2, beams=2, max_len=8, page_size=2, vocab=10)
    with pytest.raises(ValueError):
        eng.BeamDecode(None, end_token=end_token, **size)
    d = eng.BeamDecode(None, end_token=9, **size)
    d.start(dev([1, 1]), 2)
    d.first(torch.zeros((2, 10), device="cuda"))
    assert status() == 0
