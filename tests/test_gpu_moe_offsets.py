"""Expert sorting with an offsets tensor longer than experts + 1: the calls
that read it find the rows in use at its end, so that the padding is zeroed."""
import pytest
import torch

from tests import rowop_reference as R
from tests.gpu_helpers import DEV
from tests.test_gpu_rowops import F, choices, empty, normal  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("extra", [0, 1, 7])
@pytest.mark.parametrize("side", [False, True])
def test_longer_offsets(F, extra, side):  # noqa: F811
    tokens, k, experts, pad, cols = 50, 2, 5, 16, 72
    e = choices(3, tokens, k, experts)
    rows = F.moe_rows(tokens * k, experts, pad)
    offsets, counts, pos, src = R.sort_choices(e, experts, pad, rows)
    end = int(offsets[-1])
    got = [torch.zeros(experts + 1 + extra, dtype=torch.int32, device=DEV), empty(torch.int32, experts),
           empty(torch.int32, tokens, k), empty(torch.int32, rows)]
    x, dy = normal(1, tokens, cols).to(DEV), normal(2, tokens, cols).to(DEV)
    w = normal(3, tokens, k, dtype=torch.float32).to(DEV)
    xs, dys = (torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dw, ed, ws = empty(torch.float32, tokens, k), e.to(DEV), F.moe_workspace(tokens * k, experts)
    torch.cuda.synchronize()
    s = torch.cuda.Stream() if side else None
    F.fp8_moe_sort(ed, experts, pad, *got, stream=s, workspace=ws)
    F.fp8_moe_dispatch(x, got[2], got[3], got[0], xs, stream=s)
    F.fp8_moe_combine_bwd(dy, xs, w, got[2], got[3], got[0], dys, dw, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got[0][:experts + 1].cpu(), offsets)
    assert (got[0][experts:] == end).all()
    assert torch.equal(got[3].cpu(), src)
    padding = (src < 0)
    for t in (xs.cpu(), dys.cpu()):
        assert not t[:end][padding[:end]].any() and (t[end:] == 7.0).all()
