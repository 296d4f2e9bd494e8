"""The 4-bit MX cast along rows and columns, and back: bit for bit the rule in
64 bits, which rms_reference states."""
import pytest
import torch

from tests import rms_reference as M
from tests.gpu_helpers import DEV

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def F():
    from scaled_fp8_gemm_amd import fp8sg
    fp8sg.lib()
    return fp8sg


def u8(*shape):
    return torch.full(shape, 0xa5, dtype=torch.uint8, device=DEV)


def cast(F, x, both=True):
    r, c = x.shape
    q, s, qT, sT = u8(r, c // 2), u8(r, c // 32), u8(c, r // 2), u8(c, r // 32)
    if both:
        F.fp8_quantize_mx4_t(x, q, s, qT, sT)
        return q, s, qT, sT
    F.fp8_quantize_mx4(x, q, s)
    return q, s


def check(q, s, x, label):
    code, byte = M.mx4(x)
    assert torch.equal(s.cpu().long(), byte), label
    assert torch.equal(q.cpu(), M.pack(code)), label


def sample(rows, cols, seed=0):
    g = torch.Generator().manual_seed(seed + rows * 7 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp2(
        torch.randint(-12, 12, (rows, cols), generator=g).float())
    return x.to(BF)


# one block, ragged ends of a tile, of a workgroup's pieces, several of each
@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 64), (1, 4096), (7, 96), (33, 160), (129, 288),
                                       (1000, 1056), (4100, 544)])
def test_along_rows(F, rows, cols):
    x = sample(rows, cols)
    check(*cast(F, x.to(DEV), False), x, "rows")


@pytest.mark.parametrize("rows,cols", [(32, 32), (32, 4096), (64, 96), (96, 160), (160, 32),
                                       (128, 128), (288, 416), (1056, 544)])
def test_both_ways(F, rows, cols):
    x = sample(rows, cols)
    q, s, qT, sT = cast(F, x.to(DEV))
    check(q, s, x, "rows")
    check(qT, sT, x.t().contiguous(), "columns")
    oT, osT = u8(cols, rows // 2), u8(cols, rows // 32)      # the columns alone
    F.fp8_quantize_mx4_t(x.to(DEV), None, None, oT, osT)
    assert torch.equal(oT, qT) and torch.equal(osT, sT)


@pytest.mark.parametrize("rows,cols", [(8160, 2080), (2048, 8192), (131072, 160), (32, 65568)])
def test_both_ways_of_large_tensors(F, rows, cols):
    """Tall tiles, whole and cut off at both edges: as the cast along rows, of
    x and of x^T."""
    x = sample(rows, cols).to(DEV)
    x[5, 7], x[rows - 1, cols - 1], x[rows // 2, 0] = float("nan"), float("inf"), -float("inf")
    x[:, 32:64] = 0
    q, s, qT, sT = cast(F, x)
    for got, want in zip((q, s, qT, sT), cast(F, x, False) + cast(F, x.t().contiguous(), False)):
        assert torch.equal(got, want)
    oT, osT = u8(cols, rows // 2), u8(cols, rows // 32)
    F.fp8_quantize_mx4_t(x, None, None, oT, osT)
    assert torch.equal(oT, qT) and torch.equal(osT, sT)


def test_every_value(F):
    """Every BF16 value beside one that gives its block a scale: alone, where
    it is the largest, and under larger ones, ties among them."""
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    for other in (0.0, 1.0, 6.0, 6.03125, 2.0 ** -126, 2.0 ** -133, 3e38, -1.5, 2.0 ** 120):
        x = torch.zeros(65536, 32, dtype=BF)
        x[:, 0] = other
        x[:, 17] = every
        check(*cast(F, x.to(DEV), False), x, str(other))
    # neighbours in one block: ties to even at every step of the grid
    x = (torch.arange(64 * 32).float() / 128 - 8).view(64, 32).to(BF)
    x[:, 0] = 6
    check(*cast(F, x.to(DEV), False), x, "ties")


def test_blocks_without_a_scale(F):
    x = sample(64, 128)
    x[3, 5], x[7, 127], x[40:44, 64:96] = float("inf"), float("nan"), 0.0
    x[9, 0:32], x[10, 32:64] = float("-inf"), -0.0
    q, s, qT, sT = cast(F, x.to(DEV))
    check(q, s, x, "rows")
    check(qT, sT, x.t().contiguous(), "columns")
    y = torch.empty(64, 128, dtype=BF, device=DEV)
    F.fp8_dequantize_mx4(q, s, 64, 128, y)
    bad = torch.isnan(y.cpu())
    assert bad[3, :32].all() and bad[7, 96:].all() and bad[9, :32].all() and bad.sum() == 96


@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 96), (16, 4096), (1100, 1056)])
def test_back(F, rows, cols):
    """Every code under every scale byte."""
    g = torch.Generator().manual_seed(rows)
    q = torch.randint(0, 256, (rows, cols // 2), generator=g).to(torch.uint8)
    s = torch.randint(0, 256, (rows, cols // 32), generator=g).to(torch.uint8)
    y = torch.full((rows, cols), 7.0, dtype=BF, device=DEV)
    F.fp8_dequantize_mx4(q.to(DEV), s.to(DEV), rows, cols, y)
    want = M.mx4_values(q, s)
    want = torch.where(want.abs() >= 2.0 ** 128, want.sign() * float("inf"), want)
    got = y.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = ~torch.isnan(want)
    assert torch.equal(got[ok], want[ok])
    assert torch.equal(torch.signbit(got[ok]), torch.signbit(want[ok]))


def test_stream_and_graph(F):
    x = sample(288, 416).to(DEV)
    want = cast(F, x)
    side, got = torch.cuda.Stream(), [torch.zeros_like(t) for t in want]
    torch.cuda.synchronize()
    F.fp8_quantize_mx4_t(x, *got, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    y, graph = torch.empty_like(x), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        F.fp8_quantize_mx4_t(x, *got)
        F.fp8_dequantize_mx4(got[0], got[1], 288, 416, y)
    for i in range(3):
        for t in got:
            t.fill_(i)
        graph.replay()
        cast(F, x)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        assert torch.equal(y.cpu().double(), M.mx4_values(want[0], want[1]))


def test_more_than_2_31_elements(F):
    rows, cols = (1 << 31) // 8192 + 32, 8192
    x = torch.randn(rows, cols, device=DEV, dtype=BF)
    q, s, qT, sT = cast(F, x)
    tail = x[-32:].cpu()
    check(q[-32:], s[-32:], tail, "rows")
    code, byte = M.mx4(tail.t().contiguous())
    assert torch.equal(sT[:, -1].cpu().long(), byte[:, 0])
    assert torch.equal(qT[:, -16:].cpu(), M.pack(code))
    q2, s2 = cast(F, x, False)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    y = torch.empty_like(x)
    F.fp8_dequantize_mx4(q, s, rows, cols, y)
    assert torch.equal(y[-32:].cpu().double(), M.mx4_values(q[-32:], s[-32:]))
