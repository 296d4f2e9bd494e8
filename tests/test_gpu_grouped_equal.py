"""Products by expert: equal calls give equal bits, on every tile."""
import pytest
import torch

from tests import grouped_reference as G
from tests.gpu_helpers import DEV
from tests.grouped_reference import BLOCK, E2M1, MX, SQUARE, TENSOR
from tests.test_gpu_grouped import fprop, segments
from tests.test_gpu_grouped_tiles import DEPTH, ROWS, rounded

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def F():
    from scaled_fp8_gemm_amd import fp8sg
    fp8sg.lib()
    return fp8sg


@pytest.mark.parametrize("tile", list(ROWS))
@pytest.mark.parametrize("sa,sb,fa,fb,k", [(TENSOR, TENSOR, 1, 0, 528), (BLOCK, SQUARE, 0, 0, 640),
                                           (BLOCK, BLOCK, 0, 0, 640), (MX, MX, 0, 0, 640),
                                           (MX, MX, 0, 0, 672), (MX, MX, 0, E2M1, 640),
                                           (MX, MX, E2M1, E2M1, 672)])
def test_equal_calls_give_equal_bits(F, tile, sa, sb, fa, fb, k):
    """Again, on another stream, and with everything elsewhere in memory."""
    lengths, n = ROWS[tile]
    n = rounded(n, sb)
    offsets, rows = segments(lengths, 0, 3)
    e = len(lengths)
    x, w = G.operand(1, rows, k, fa, sa), G.operand(2, e * n, k, fb, sb, tensors=e)
    first = fprop(F, x, w, offsets, e, rows, n, k, sa, sb, fa, fb)
    held = [t.to(DEV) for t in (*x, *w)]         # where the first call's operands were
    assert torch.equal(first, fprop(F, x, w, offsets, e, rows, n, k, sa, sb, fa, fb))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = fprop(F, x, w, offsets, e, rows, n, k, sa, sb, fa, fb)
    side.synchronize()
    assert torch.equal(first, other) and len(held) == 4


@pytest.mark.parametrize("tile", list(DEPTH))
@pytest.mark.parametrize("scaling", [TENSOR, BLOCK, MX])
def test_equal_gradients(F, tile, scaling):
    lengths, n, k = DEPTH[tile]
    offsets, rows = segments([v * 128 for v in lengths])
    e = len(lengths)
    off = torch.tensor(offsets, dtype=torch.int32, device=DEV)
    a, b = (F.operand(q.to(DEV), 0, scaling, s.to(DEV)) for q, s in
            (G.operand(3, n, rows, 0, scaling), G.operand(4, k, rows, 0, scaling)))
    out = []
    for _ in range(3):
        out.append(torch.full((e, n, k), -777.0, dtype=BF, device=DEV))
        F.fp8_gemm_grouped_wgrad(a, b, off, e, rows, n, k, out[-1])
    assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])
