"""A row's sums are the same bits in all of its lanes: columns that hold the
same values give the same bits, wherever in the row they are."""
import pytest
import torch

from tests.gpu_helpers import DEV
from tests.test_gpu_rowops import F, empty, normal  # noqa: F401

pytestmark = pytest.mark.gpu

# rows of one wave (one and two slots a lane), of several waves
WIDTHS = [64, 128, 264, 512, 520, 1024, 1032, 4096, 12288]


@pytest.mark.parametrize("cols", WIDTHS)
def test_equal_columns_have_equal_results(F, cols):  # noqa: F811
    rows = 400
    # a mean that is large against the spread: an ulp of it shows
    x = 1000.3 + 0.01 * normal(cols, rows, cols, dtype=torch.float32)
    dy = normal(cols + 1, rows, cols)
    x[:, ::8], dy[:, ::8] = x[:, :1].clone(), dy[:, :1].clone()    # one column of every slot
    x, dy = x.to(DEV), dy.to(DEV)
    one, zero = torch.ones(cols, device=DEV), torch.zeros(cols, device=DEV)
    y, dx = empty(torch.bfloat16, rows, cols), empty(torch.float32, rows, cols)
    mo, ro = empty(torch.float32, rows), empty(torch.float32, rows)
    dg, db = empty(torch.float32, cols), empty(torch.float32, cols)
    F.fp8_layernorm_fwd(x, one, zero, 1e-5, y, mo, ro)
    F.fp8_layernorm_bwd(dy, x, mo, ro, one, dx, dg, db)
    for name, t in (("y", y), ("dx", dx)):
        t = t[:, ::8]
        assert torch.equal(t, t[:, :1].expand_as(t)), name
    for name, t in (("dgamma", dg[::8]), ("dbeta", db[::8])):
        assert torch.equal(t, t[:1].expand_as(t)), name
