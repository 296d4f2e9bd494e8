"""GPU parity of the dense GEMMs with 4-bit operands: every tile size, depths
that end inside a step, the FP32 and fused epilogues."""
import pytest
import torch

from tests import grouped_reference as G
from tests.gpu_helpers import DEV
from tests.grouped_reference import E2M1, MX
from tests.test_gpu_grouped import some_columns

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def F():
    from scaled_fp8_gemm_amd import fp8sg
    fp8sg.lib()
    return fp8sg


def operands(F, m, n, k, fa, spoil=None):
    a, b = G.operand(m + k, m, k, fa, MX), G.operand(n + k + 1, n, k, E2M1, MX)
    if spoil:
        spoil(a, b)
    dev = [F.operand(q.to(DEV), f, MX, s.to(DEV)) for (q, s), f in ((a, fa), (b, E2M1))]
    return dev, G.values(*a, fa, MX), G.values(*b, E2M1, MX)


FORMATS = [0, 1, E2M1]
# one row and more than a tile's
ROWS = [1, 16, 17, 33, 64, 65, 130, 390, 520]
# (rows, columns) of the tiles that need many columns: 64 x 128, 128, 256
WIDE = [(130, 6800), (300, 10900), (520, 13907)]


@pytest.mark.parametrize("m", ROWS)
@pytest.mark.parametrize("n", [1, 40, 259])
@pytest.mark.parametrize("fa", FORMATS)
def test_sizes(F, orc, m, n, fa):
    for k in (160, 384) if m < 300 else (128, 96):
        (a, b), av, bv = operands(F, m, n, k, fa)
        y = torch.full((m, n), -777.0, dtype=BF, device=DEV)
        F.fp8_gemm_fprop(a, b, m, n, k, y)
        G.check(orc, y, av, bv, f"{k}")


@pytest.mark.parametrize("m,n", WIDE)
@pytest.mark.parametrize("k", [32, 160, 256, 384, 640])
@pytest.mark.parametrize("fa", FORMATS)
def test_wide(F, orc, m, n, k, fa):
    (a, b), av, bv = operands(F, m, n, k, fa)
    y = torch.full((m, n), -777.0, dtype=BF, device=DEV)
    F.fp8_gemm_fprop(a, b, m, n, k, y)
    cols = some_columns(n)
    G.check(orc, y[:, cols].contiguous(), av, bv[cols], "fprop")


@pytest.mark.parametrize("k", [32, 64, 96, 128, 256, 288, 512, 544, 640, 1024, 1056, 4096, 4640])
@pytest.mark.parametrize("m", [3, 28, 140])
@pytest.mark.parametrize("fa", FORMATS)
def test_depths(F, orc, m, k, fa):
    (a, b), av, bv = operands(F, m, 35, k, fa)
    y = torch.full((m, 35), -777.0, dtype=BF, device=DEV)
    F.fp8_gemm_fprop(a, b, m, 35, k, y)
    G.check(orc, y, av, bv, "fprop")


@pytest.mark.parametrize("m", [5, 40, 140, 400])
@pytest.mark.parametrize("k", [32, 128, 160, 384, 640])
@pytest.mark.parametrize("fa", FORMATS)
def test_nan_scales_stay_in_their_row(F, orc, m, k, fa):
    def spoil(a, b):
        a[1][1, 0] = a[1][4, -1] = 255
        b[1][2, 0] = b[1][7, -1] = b[1][-1, -1] = 255
    (a, b), av, bv = operands(F, m, 40, k, fa, spoil)
    y = torch.zeros(m, 40, dtype=BF, device=DEV)
    F.fp8_gemm_fprop(a, b, m, 40, k, y)
    G.check(orc, y, av, bv, "fprop")


@pytest.mark.parametrize("fa", FORMATS)
def test_unaligned_scales(F, orc, fa):
    """E8M0 scales that start at any byte."""
    for m in (5, 140):
        (a, b), av, bv = operands(F, m, 40, 512, fa)
        y = [torch.zeros(m, 40, dtype=BF, device=DEV) for _ in range(2)]
        F.fp8_gemm_fprop(a, b, m, 40, 512, y[0])
        moved = []
        for o in (a, b):
            s = o._tensors[1].reshape(-1)
            buf = torch.full((s.numel() + 3,), 255, dtype=torch.uint8, device=DEV)
            buf[3:] = s
            moved.append(F.operand(o._tensors[0], o.fmt, MX, buf[3:]))
        F.fp8_gemm_fprop(*moved, m, 40, 512, y[1])
        assert torch.equal(*y)
        G.check(orc, y[1], av, bv, "moved")


@pytest.mark.parametrize("m,n,k", [(7, 40, 160), (150, 72, 256), (400, 33, 128)])
def test_dgrad_and_wgrad(F, orc, m, n, k):
    """The other two products of a layer: dgrad contracts N, wgrad M."""
    for fa in (1, E2M1):
        (a, b), av, bv = operands(F, m, k, n // 32 * 32, fa)
        dx = torch.zeros(m, k, dtype=BF, device=DEV)
        F.fp8_gemm_dgrad(a, b, m, n // 32 * 32, k, dx)
        G.check(orc, dx, av, bv, "dgrad")
    mm = (m + 31) // 32 * 32
    (a, b), av, bv = operands(F, n, k, mm, E2M1)
    dw = torch.zeros(n, k, dtype=BF, device=DEV)
    F.fp8_gemm_wgrad(a, b, mm, n, k, dw)
    G.check(orc, dw, av, bv, "wgrad")


@pytest.mark.parametrize("m,n", [(5, 16), (5, 41), (28, 272), (140, 41), (400, 272)] + WIDE)
def test_f32_out(F, m, n):
    cols = some_columns(n)
    for fa in FORMATS:
        (a, b), av, bv = operands(F, m, n, 160, fa)
        dw = torch.full((m, n), 5.0, device=DEV)
        F.fp8_gemm_wgrad_f32(a, b, 160, m, n, dw)
        G.check_f32(dw[:, cols], torch.zeros(m, len(cols)), av, bv[cols], "stored")
        first = dw.clone()
        F.fp8_gemm_wgrad_f32(a, b, 160, m, n, dw, accumulate=True)
        assert torch.equal(dw, first + first)


@pytest.mark.parametrize("m,n", [(1, 16), (30, 272), (140, 272), (130, 6800), (300, 10912),
                                 (520, 13904)])
@pytest.mark.parametrize("y_fmt", [0, 1])
def test_fused(F, m, n, y_fmt):
    """The fused cast and amax are those of the BF16 output."""
    for fa in FORMATS:
        (a, b), _, _ = operands(F, m, n, 256, fa)
        y, want = (torch.zeros(m, n, dtype=BF, device=DEV) for _ in range(2))
        F.fp8_gemm_fprop(a, b, m, n, 256, want)
        s, ws = torch.full((1,), 0.37, device=DEV), F.workspace()
        q, amax = torch.zeros(m, n, dtype=torch.uint8, device=DEV), torch.zeros(1, device=DEV)
        F.fp8_gemm_fprop_fused(a, b, m, n, 256, y, y_fmt, s, q, amax, workspace=ws)
        wq, wa = torch.zeros_like(q), torch.zeros_like(amax)
        F.fp8_quantize_tensor(want, y_fmt, s, wq, None, wa, workspace=ws)
        assert torch.equal(y, want) and torch.equal(q, wq) and torch.equal(amax, wa)
        q2 = torch.zeros_like(q)
        F.fp8_gemm_fprop_fused(a, b, m, n, 256, None, y_fmt, s, q2, None)    # the cast alone
        assert torch.equal(q2, wq)


def test_empty(F):
    for m, n in ((0, 16), (16, 0)):
        (a, b), _, _ = operands(F, m, n, 64, 0)
        amax = torch.full((1,), 3.0, device=DEV)
        F.fp8_gemm_fprop_fused(a, b, m, n, 64, torch.empty(m, n, dtype=BF, device=DEV), 0, None,
                               None, amax, workspace=F.workspace())
        assert amax.item() == 0
    for m in (3, 200):
        (a, b), _, _ = operands(F, m, 16, 0, 0)
        y = torch.full((m, 16), 3.0, dtype=BF, device=DEV)
        F.fp8_gemm_fprop(a, b, m, 16, 0, y)
        assert (y == 0).all()


def test_cast_then_product(F, orc):
    """The 4-bit cast's own outputs, both ways, as operands."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(70, 288, generator=g).bfloat16().to(DEV)
    w = torch.randn(96, 288, generator=g).bfloat16().to(DEV)
    u = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    xq, xs, wq, ws, wT, wTs = u(70, 144), u(70, 9), u(96, 144), u(96, 9), u(288, 48), u(288, 3)
    F.fp8_quantize_mx4(x, xq, xs)
    F.fp8_quantize_mx4_t(w, wq, ws, wT, wTs)
    y = torch.zeros(70, 96, dtype=BF, device=DEV)
    F.fp8_gemm_fprop(F.operand(xq, E2M1, MX, xs), F.operand(wq, E2M1, MX, ws), 70, 96, 288, y)
    G.check(orc, y, G.values(xq, xs, E2M1, MX), G.values(wq, ws, E2M1, MX), "fprop")
    yq, ys, dx = u(70, 96), u(70, 3), torch.zeros(70, 288, dtype=BF, device=DEV)
    F.fp8_quantize_mx(y, F.E5M2, yq, ys)
    F.fp8_gemm_dgrad(F.operand(yq, 1, MX, ys), F.operand(wT, E2M1, MX, wTs), 70, 96, 288, dx)
    G.check(orc, dx, G.values(yq, ys, 1, MX), G.values(wT, wTs, E2M1, MX), "dgrad")


def test_deterministic_and_captured(F):
    for m in (3, 200):
        (a, b), _, _ = operands(F, m, 300, 4096, E2M1)
        y = [torch.zeros(m, 300, dtype=BF, device=DEV) for _ in range(2)]
        F.fp8_gemm_fprop(a, b, m, 300, 4096, y[0])
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        F.fp8_gemm_fprop(a, b, m, 300, 4096, y[1], stream=side)
        side.synchronize()
        assert torch.equal(*y)
        with torch.cuda.graph(graph):
            F.fp8_gemm_fprop(a, b, m, 300, 4096, y[1])
        for _ in range(3):
            y[1].zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(*y)
