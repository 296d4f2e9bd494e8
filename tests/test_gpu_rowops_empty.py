"""Row operators on tensors without rows, at widths on both sides of every
change in how rows are dealt out: amax 0, gradients of gamma and beta zero."""
import pytest
import torch

from tests.gpu_helpers import DEV
from tests.test_gpu_rowops import BLOCK, F, TENSOR, empty  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols", [1, 40, 4097, 8192, 8193, 12288, 12289, 16384, 16385, 32768])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("held", [False, True])
def test_layernorm_without_rows_at_any_width(F, cols, xt, held):  # noqa: F811
    x = torch.empty((0, cols), dtype=xt, device=DEV)
    y = torch.empty((0, cols), dtype=torch.bfloat16, device=DEV)
    w, e = torch.ones(cols, device=DEV), torch.empty(0, device=DEV)
    q = torch.empty((0, cols), dtype=torch.uint8, device=DEV)
    amax, scale = empty(torch.float32, 1), torch.ones(1, device=DEV)
    F.fp8_layernorm_fwd(x, w, w, 1e-5, y, e, e, yq=F.cast_out(q, 0, TENSOR, None, scale, amax))
    assert amax.item() == 0
    dg, db = empty(torch.float32, cols), empty(torch.float32, cols)
    if held:
        F.fp8_layernorm_bwd(y, None, None, e, w, x, dg, db, xhat=F.operand(q, 0, BLOCK, e))
    else:
        F.fp8_layernorm_bwd(y, x, e, e, w, x, dg, db)
    assert not dg.any() and not db.any()
