"""The fused 4-bit product whose small tiles are more than the workspace has
words for their maxima: it takes the largest tile, and writes nothing of the
workspace but those words."""
import pytest
import torch

from tests.gpu_helpers import DEV
from tests.grouped_reference import E2M1, MX
from tests.test_seg_shape import tile  # noqa: F401  (a fixture)

BF = torch.bfloat16
WORDS = 1 << 16                       # of maxima
# rows, columns: one tile more than the words, and as many as them
SIZES = [(1, 64 * WORDS + 16), (30, 64 * WORDS + 16), (1, 64 * WORDS)]


@pytest.mark.parametrize("m,n", SIZES)
def test_tile(tile, m, n):  # noqa: F811
    small = "16x64" if m <= 24 else "32x64"
    assert tile("rows", m, n, 1, False, True, 0) == small
    assert tile("rows", m, n, 1, False, True, WORDS) == ("256x256" if n > 64 * WORDS else small)


@pytest.mark.gpu
@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("fa", [0, E2M1])
def test_maxima_fit_the_workspace(m, n, fa):
    from scaled_fp8_gemm_amd import fp8sg as F
    g = torch.Generator(device=DEV).manual_seed(m)
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=DEV,  # noqa: E731
                                            dtype=torch.uint8)
    a = F.operand(byte(0, 0x7f, m, 32 // (2 if fa == E2M1 else 1)), fa, MX, byte(120, 128, m, 1))
    b = F.operand(byte(0, 256, n, 16), E2M1, MX, byte(110, 120, n, 1))
    b._tensors[1][-1] = 126           # the largest output is of the last tile
    memory = torch.full((F.WORKSPACE_BYTES + 4096,), 77, dtype=torch.uint8, device=DEV)
    ws = memory[:F.WORKSPACE_BYTES]
    F.fp8_workspace_init(ws)
    before = memory.clone()
    want, y = (torch.zeros(m, n, dtype=BF, device=DEV) for _ in range(2))
    F.fp8_gemm_fprop(a, b, m, n, 32, want)
    s, amax = torch.full((1,), 0.37, device=DEV), torch.zeros(1, device=DEV)
    q = torch.zeros(m, n, dtype=torch.uint8, device=DEV)
    F.fp8_gemm_fprop_fused(a, b, m, n, 32, y, F.E4M3, s, q, amax, workspace=ws)
    assert torch.equal(memory[WORDS * 4:], before[WORDS * 4:])
    assert torch.equal(y, want) and amax.item() == want.abs().amax().item()
    wq = torch.zeros_like(q)
    F.fp8_quantize_tensor(want, F.E4M3, s, wq)
    assert torch.equal(q, wq)
