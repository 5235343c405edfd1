"""Workspaces of the training operators: what is taken for the largest call serves every smaller
one.  Host logic, no GPU."""
import pytest

eng = pytest.importorskip("hashed_gram_memory_tid2eid_amd")


def steps(dim, most):
    """Place counts around which the length of a chunk changes (a chunk's lanes each sum 8 columns,
    padded to whole groups of 32 to 2,048), and a spread of others."""
    group = next(g for g in (32, 64, 128, 256, 512, 1024, 2048) if g >= dim or g == 2048)
    lanes = -(-dim // group) * group // 8
    near = {ch * 131072 // lanes + d for ch in (4, 8, 16, 32) for d in range(-33, 34)}
    return sorted(n for n in near | set(range(1, 200)) | {most * i // 97 for i in range(1, 98)} if 1 <= n <= most)


@pytest.mark.parametrize("dim", [1, 24, 96, 128, 256, 538, 1024, 2056, 4096, 6500])
def test_gradient_workspace_serves_fewer_places(dim):
    ns = steps(dim, 6_000_000 * 32 // max(dim, 32))
    sizes = [eng.engram_embed_grad_workspace(n, 1000, dim) for n in ns]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


@pytest.mark.parametrize("max_tokens", [1365, 1400, 1536, 1900, 2731, 5462])
@pytest.mark.parametrize("cols, dim", [(24, 256), (6, 128), (3, 6500)])
def test_every_smaller_call_fits(cols, dim, max_tokens):
    most = eng.engram_embed_grad_workspace(max_tokens * cols, 1000, dim)
    assert all(eng.engram_embed_grad_workspace(T * cols, 1000, dim) <= most for T in range(1, max_tokens))


def test_gradient_of_columns_past_32_bits_is_refused():
    """Columns rounded up to whole groups of lanes have to fit 32 bits: the kernels count them so."""
    widest = 2 ** 31 - 2048
    assert eng.engram_embed_grad_workspace(1, 1, widest) > 0
    work, P = 1 << 40, 1 << 20  # an aligned address that nothing reads
    for dim in (widest + 1, 2 ** 31 - 1):
        with pytest.raises(eng.EngramError):
            eng.engram_embed_grad_workspace(1, 1, dim)
        for mode in (0, 1, 2):
            assert eng._lib.engram_embed_grad(P, 1, 1, 1, 1, dim, 1.0, P, eng.ENGRAM_DTYPE_BF16, dim, dim, mode, P,
                                              eng.ENGRAM_DTYPE_F32, dim, P, P, P, work, None) == \
                eng.STATUS["ENGRAM_E_UNSUPPORTED"]


@pytest.mark.parametrize("dim, lanes", [(122, 16), (256, 32), (4093, 512), (4096, 512)])
def test_chunks_grow_where_enough_lanes_are_left(dim, lanes):
    """A longer chunk halves the partial rows, so the workspace stays where it was for a while."""
    for chunk in (8, 16, 32):
        n = chunk * 131072 // lanes
        before, last, first, behind = (eng.engram_embed_grad_workspace(m, 1000, dim) for m in (n - 64, n - 1, n, n + n // 4))
        assert before < last == first == behind
