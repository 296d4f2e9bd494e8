"""Layer norm of FP32 rows whose mean is large against their spread.

A rounded sum is off by 64 U sum |v| (U = 2^-24), as in rowop_reference; the
mean of the deviations d from a first mean corrects it, so what is left is the
mean's own half step, U |mean|, and 64 roundings of sums of deviations, which
are the row's own and the first mean's error of at most 70 U of the values:
75 U (mean |d| + 70 U mean |x|).  A row of one value has deviations of the
same bits throughout; their mean is within 70 U of them, which is far below
half a step of the value, so its mean is that value and its normalised row 0."""
import pytest
import torch

from tests import rowop_reference as R
from tests.gpu_helpers import DEV, bytes8
from tests.test_gpu_rowops import BLOCK, F, MX, empty, make_cast, normal  # noqa: F401

pytestmark = pytest.mark.gpu

# values of no few bits, at every way of dealing out a row
WIDTHS = [1, 5, 129, 512, 700, 1003, 2049, 4096, 6144, 8193, 12288, 16384, 20000, 32768]
VALUES = [18999.457, 1779.9448, 152.34348, 0.1, -333.33334, 1e6 + 0.0625 * 3]


@pytest.mark.parametrize("cols", WIDTHS)
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
def test_rows_of_one_value(F, cols, xt):  # noqa: F811
    x = torch.tensor(VALUES).to(xt)[:, None].expand(-1, cols).contiguous()
    beta = normal(cols, cols, dtype=torch.float32)
    rows = len(VALUES)
    y, mo, ro = (empty(torch.bfloat16, rows, cols), empty(torch.float32, rows),
                 empty(torch.float32, rows))
    cq, cs, ck = make_cast(F, rows, cols, BLOCK)
    F.fp8_layernorm_fwd(x.to(DEV), torch.ones(cols, device=DEV), beta.to(DEV), 1e-5, y, mo, ro,
                        xhat=ck)
    assert torch.equal(mo.cpu(), x[:, 0].float())
    # 1 / sqrt(eps): a square root and a quotient of the FP32 eps
    want = 1 / torch.sqrt(torch.full((rows,), 1e-5).double())
    R.check_close(ro, want, 4 * R.U * want, "rstd")
    assert not (bytes8(cq) & 0x7f).any() and (cs == 1).all()
    assert torch.equal(y.cpu(), beta.bfloat16().expand(rows, -1))


@pytest.mark.parametrize("cols", [c for c in WIDTHS if c > 100])
@pytest.mark.parametrize("mean,spread", [(18999.457, 0.5), (152.34348, 0.01), (-1e5, 3.0),
                                         (0.3, 1.0)])
def test_rows_with_a_large_mean(F, cols, mean, spread):  # noqa: F811
    rows = 7
    x = mean + spread * normal(cols, rows, cols, dtype=torch.float32)
    gamma = 1 + 0.2 * normal(1, cols, dtype=torch.float32)
    beta = normal(2, cols, dtype=torch.float32, scale=0.1)
    xd = [v.double() for v in (x, gamma, beta)]
    m, rstd, xhat, y = R.ln_fwd(*xd, 1e-5)
    d = (xd[0] - m[:, None]).abs().mean(1)
    tm = 1.01 * R.U * m.abs() + 75 * R.U * (d + 70 * R.U * xd[0].abs().mean(1))
    # as ln_fwd_bounds, with this bound of the mean
    rel = 40 * R.U + rstd * tm + (rstd * tm) ** 2
    th = xhat.abs() * (rel + 4 * R.U)[:, None] + (rstd * tm * 1.01)[:, None]
    ty = xd[1].abs() * th + 3 * R.U * ((xhat * xd[1]).abs() + xd[2].abs())
    yo, mo, ro = (empty(torch.bfloat16, rows, cols), empty(torch.float32, rows),
                  empty(torch.float32, rows))
    q, s, yq = make_cast(F, rows, cols, MX)
    cq, cs, ck = make_cast(F, rows, cols, BLOCK)
    F.fp8_layernorm_fwd(x.to(DEV), gamma.to(DEV), beta.to(DEV), 1e-5, yo, mo, ro, yq=yq, xhat=ck)
    R.check_close(mo, m, tm, "mean")
    R.check_close(ro, rstd, rstd * rel, "rstd")
    R.check_bf16(yo, y, ty, "y")
    R.check_cast(q, s, y, ty, 0, MX, "yq")
    R.check_cast(cq, cs, xhat, th, 0, BLOCK, "xhat")


def test_an_infinite_value_keeps_the_mean_infinite(F):  # noqa: F811
    x = normal(5, 2, 1000, dtype=torch.float32)
    x[1, 3] = float("-inf")
    y, mo, ro = empty(torch.bfloat16, 2, 1000), empty(torch.float32, 2), empty(torch.float32, 2)
    w = torch.ones(1000, device=DEV)
    F.fp8_layernorm_fwd(x.to(DEV), w, w, 1e-5, y, mo, ro)
    assert mo[1].item() == float("-inf") and torch.isnan(y[1]).all()
    assert torch.isfinite(y[0]).all() and torch.isfinite(mo[0])
