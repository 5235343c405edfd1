"""The quantiser's blocks where a code is decided by the quotient's last bit, and rows alone in many tiles.
Codes and scales follow from single correctly rounded operations: compared bit for bit."""
import pytest
import torch

from test_gpu_train_ops import BF16, DEV, F32, eng, gen, held, quantize_ref, rough, up  # noqa: F401  (eng is a fixture)

pytestmark = pytest.mark.gpu


def on_ties(g, M, K, block, exponent):
    """x [M][K] in blocks of block x 128: values that lie, as nearly as fp32 can say, half way between two
    codes of their block's scale, which is 1 to 2 times 2^exponent; and the block's largest."""
    s = (1 + torch.rand((M // block, 1, K // 128, 1), generator=g, device=DEV, dtype=torch.float64)) * 2.0 ** exponent
    shape = (M // block, block, K // 128, 128)
    e = torch.randint(-6, 1, shape, generator=g, device=DEV).double()
    k = torch.randint(0, 8, shape, generator=g, device=DEV).double()
    tie = torch.where(k % 2 == 0, (k + 0.5) * 2.0 ** -9, (1 + (2 * k + 1) / 16) * torch.exp2(e))
    most = (448 * s[:, 0, :, 0]).float()
    # the scale that the largest gives, to its last bit (on the host: one rounding)
    own = torch.maximum(most.cpu() / torch.tensor(448.0), torch.tensor(2.0 ** -126)).double().to(DEV)
    x = (tie * own[:, None, :, None]).float()
    x[:, 0, :, 0] = most
    return (x * torch.where(torch.rand(shape, generator=g, device=DEV) < 0.5, -1.0, 1.0)).view(M, K)


@pytest.mark.parametrize("exponent", [-126, -124, -120, -116, -112, -108, -100, -80, -65, -64, -63, -20, 0, 60, 110])
@pytest.mark.parametrize("e8m0", [False, True])
@pytest.mark.parametrize("block", [1, 128])
def test_quotients_on_ties(eng, exponent, e8m0, block):
    """Blocks of every size down to the smallest scale, along the rows and along the columns, in every
    combination of outputs."""
    M, K = 256, 512
    x = on_ties(gen(exponent + 1000), M, K, block, exponent)
    kind = torch.uint8 if e8m0 else F32
    for values, transposed in ((x, False), (x.t().contiguous(), True)):
        m, k = values.shape
        refs = quantize_ref(values, e8m0, block), quantize_ref(values.t(), e8m0, block)
        for rows, cols in ((True, True), (True, False), (False, True)):
            q, qt = (torch.empty(n, dtype=torch.float8_e4m3fn, device=DEV) for n in ((m, k), (k, m)))
            s, st = (torch.empty(r[1].shape, dtype=kind, device=DEV) for r in refs)
            eng.engram_fp8_quantize(values, q if rows else None, s if rows else None, q_t=qt if cols else None,
                                    scales_t=st if cols else None, block_rows=block)
            for wanted, codes, scales, (wq, ws) in ((rows, q, s, refs[0]), (cols, qt, st, refs[1])):
                if wanted:
                    assert torch.equal(scales.cpu(), held(ws, e8m0))
                    assert torch.equal(codes.cpu().float(), wq.float())


def test_small_blocks_beside_large_and_empty_ones(eng):
    """Rows of one tile whose scales lie on both sides of where the division changes."""
    g = gen(77)
    sizes = [-126, -110, -64, -65, 0, 30, -90, -63]
    x = torch.stack([on_ties(g, 16, 256, 1, e) for e in sizes], 1).view(128, 256)  # rows take turns
    x[5] = 0.0
    q, qt = torch.empty((128, 256), dtype=torch.float8_e4m3fn, device=DEV), torch.empty((256, 128), dtype=torch.float8_e4m3fn, device=DEV)
    s, st = torch.empty((2, 128), device=DEV), torch.empty((1, 256), device=DEV)
    eng.engram_fp8_quantize(x, q, s, q_t=qt, scales_t=st)
    for codes, scales, values in ((q, s, x), (qt, st, x.t())):
        wq, ws = quantize_ref(values, False)
        assert torch.equal(scales.cpu(), ws) and torch.equal(codes.cpu().float(), wq.float())


@pytest.mark.parametrize("M, K", [(1344, 6130), (1345, 6130), (1400, 6130), (8192, 1024), (8193, 1024), (16_381, 700),
                                  (65_537, 130), (4000, 2049)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("e8m0", [False, True])
def test_rows_alone(eng, M, K, dtype, e8m0):
    """Tiles of 16 rows up to 2,048 tiles of 32 x 128, of 64 rows from there on: on both sides, with rows and
    columns past the last whole tile."""
    assert (-(-K // 128) * -(-M // 32) > 2048) == ((M, K) not in ((1344, 6130), (8192, 1024)))
    x = rough(gen(M + K), M, K, dtype)
    wq, ws = quantize_ref(x, e8m0)
    q = torch.full((M + 1, up(K) + 16), 9, dtype=torch.uint8, device=DEV)
    s = torch.empty(ws.shape, dtype=torch.uint8 if e8m0 else F32, device=DEV)
    eng.engram_fp8_quantize(x, q[:M], s)
    assert torch.equal(s.cpu(), held(ws, e8m0))
    assert torch.equal(q[:M, :up(K)].cpu().view(torch.float8_e4m3fn).float(), wq.float())
    assert bool((q[:M, up(K):] == 9).all()) and bool((q[M] == 9).all())
