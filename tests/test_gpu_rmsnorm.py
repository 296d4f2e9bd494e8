"""GPU parity of root-mean-square norm and the residual's addition with their
formulas in 64 bits, under the bounds of rms_reference."""
import pytest
import torch

from tests import rms_reference as M
from tests import rowop_reference as R
from tests.gpu_helpers import DEV
from tests.test_gpu_rowops import BLOCK, MX, NONE, TENSOR, empty, make_cast, normal

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def F():
    from scaled_fp8_gemm_amd import fp8sg
    fp8sg.lib()
    return fp8sg


# widths that end inside a slot, a tile, a wave's share, at and across each
# number of slots per thread, up to the limit; enough rows for several a
# workgroup
SHAPES = [(1, 1), (3, 7), (5, 8), (4, 127), (9, 129), (6, 512), (5, 513), (7, 1003), (3, 1024),
          (2, 1025), (300, 2048), (4, 2057), (3, 4096), (2, 8195), (2, 12288), (3, 16384),
          (2, 16385), (3, 20000), (2, 32768)]


def case(rows, cols, xt, wt, delta):
    x = normal(rows + cols, rows, cols, dtype=F32)
    x[:, ::97] *= 8
    d = normal(rows * 3 + cols, rows, cols, scale=0.3) if delta else None
    return x.to(xt), d, (1 + 0.2 * normal(cols, cols, dtype=F32)).to(wt)


def dev(t):
    return None if t is None else t.to(DEV)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("xt,wt,scaling,fmt,delta", [
    (BF, F32, MX, 0, True), (BF, BF, BLOCK, 1, False), (F32, F32, TENSOR, 0, True),
    (F32, BF, MX, 1, False), (BF, BF, NONE, 0, True), (F32, F32, BLOCK, 0, True)])
def test_forward(F, shape, xt, wt, scaling, fmt, delta):
    rows, cols = shape
    x, d, gamma = case(rows, cols, xt, wt, delta)
    h = M.stream(x, d)
    rstd, xhat, y = M.rms_fwd(h.double(), gamma.double(), 1e-5)
    tr, th, ty = M.rms_fwd_bounds(rstd, xhat, y)
    ho, yo, ro = empty(xt, rows, cols), empty(BF, rows, cols), empty(F32, rows)
    scale, amax = torch.full((1,), 32.0, device=DEV), empty(F32, 1)
    q = s = yq = None
    if scaling != NONE:
        q, s, yq = make_cast(F, rows, cols, scaling, fmt, scale=scale, amax=amax)
    cq, cs, ck = make_cast(F, rows, cols, BLOCK)
    F.fp8_rmsnorm_fwd(dev(x), dev(d), dev(gamma), 1e-5, ho, yo, ro, yq=yq, xhat=ck)
    assert torch.equal(ho.cpu(), h)
    R.check_close(ro, rstd, tr, "rstd")
    R.check_bf16(yo, y, ty, "y")
    R.check_cast(cq, cs, xhat, th, 0, BLOCK, "xhat")
    if scaling != NONE:
        R.check_cast(q, s, y, ty, fmt, scaling, "yq", scale=32.0)
    if scaling == TENSOR:
        R.check_close(amax, y.abs().max(), ty.max(), "amax")


@pytest.mark.parametrize("shape", SHAPES + [(300, 264), (1100, 200), (700, 1400), (520, 5120)])
@pytest.mark.parametrize("xt,wt,held,dres", [
    (BF, F32, 0, True), (F32, BF, 0, False), (BF, BF, None, True), (F32, F32, None, True),
    (BF, F32, None, False), (F32, F32, 1, True), (BF, BF, 1, False)])
def test_backward(F, shape, xt, wt, held, dres):
    rows, cols = shape
    h, _, gamma = case(rows, cols, xt, wt, False)
    dy = normal(rows * cols, rows, cols)
    res = normal(rows * cols + 1, rows, cols, dtype=F32).to(xt) if dres else None
    ro = empty(F32, rows)
    cq, cs, ck = make_cast(F, rows, cols, BLOCK, held or 0)
    F.fp8_rmsnorm_fwd(dev(h), None, dev(gamma), 1e-5, None, None, ro, xhat=ck)
    dx, dg = empty(xt, rows, cols), empty(F32, cols)
    r, g = ro.cpu().double(), gamma.double()
    if held is not None:
        F.fp8_rmsnorm_bwd(dev(dy), None, ro, dev(gamma), dev(res), dx, dg,
                          xhat=F.operand(cq, held, F.SCALE_BLOCK_1x128, cs))
        xhat = R.held_values(cq, cs, held)
    else:
        F.fp8_rmsnorm_bwd(dev(dy), dev(h), ro, dev(gamma), dev(res), dx, dg)
        xhat = h.double() * r[:, None]
    t_xhat = M.U * xhat.abs()
    rd = None if res is None else res.double()
    wx, wg = M.rms_bwd(dy.double(), xhat, r, g, rd)
    tx, tg = M.rms_bwd_bounds(dy.double(), xhat, t_xhat, r, g, rd)
    if xt == BF:
        R.check_bf16(dx, wx, tx, "dx")
    else:
        R.check_close(dx, wx, tx + R.U * wx.abs(), "dx")
    R.check_close(dg, wg, tg, "dgamma")


@pytest.mark.parametrize("xt", [BF, F32])
def test_is_the_addition_then_the_norm(F, xt):
    """The fused call gives the bits of the addition followed by the norm."""
    x, d, gamma = (dev(t) for t in case(37, 4101, xt, F32, True))
    h, y, r = torch.empty_like(x), empty(BF, 37, 4101), empty(F32, 37)
    F.fp8_rmsnorm_fwd(x, d, gamma, 1e-6, h, y, r)
    y2, r2 = torch.empty_like(y), torch.empty_like(r)
    F.fp8_rmsnorm_fwd(h, None, gamma, 1e-6, None, y2, r2)
    assert torch.equal(y, y2) and torch.equal(r, r2)
    h3, r3 = torch.empty_like(h), torch.empty_like(r)
    F.fp8_rmsnorm_fwd(x, d, gamma, 1e-6, h3, None, r3)      # the stream alone
    assert torch.equal(h, h3) and torch.equal(r, r3)


def test_rows_without_content(F):
    """Zero rows, rows with infinities and NaN, and no rows."""
    x = torch.zeros(6, 300, dtype=BF)
    x[1, 5], x[2, 299], x[3, 0], x[4] = float("inf"), float("nan"), 1e-30, 3.0
    gamma = torch.ones(300)
    y, r = empty(BF, 6, 300), empty(F32, 6)
    F.fp8_rmsnorm_fwd(dev(x), None, dev(gamma), 1e-5, None, y, r)
    rstd, _, want = M.rms_fwd(x.double(), gamma.double(), 1e-5)
    y, r = y.cpu().double(), r.cpu().double()
    assert torch.equal(torch.isnan(y), torch.isnan(want)) and r[1] == 0 and torch.isnan(r[2])
    ok = ~torch.isnan(want)
    assert torch.allclose(y[ok], want[ok], rtol=2.0 ** -8, atol=0)
    x0 = torch.empty(0, 300, dtype=BF, device=DEV)
    F.fp8_rmsnorm_fwd(x0, None, dev(gamma), 1e-5, None, x0, empty(F32, 0))
    dg = empty(F32, 300)
    F.fp8_rmsnorm_bwd(x0, x0, empty(F32, 0), dev(gamma), None, x0, dg)
    assert torch.equal(dg.cpu(), torch.zeros(300))
    # no rows, with an amax
    amax = empty(F32, 1)
    F.fp8_rmsnorm_fwd(x0, None, dev(gamma), 1e-5, None, x0, empty(F32, 0),
                      yq=F.cast_out(empty(torch.uint8, 0, 300), 0, TENSOR, None,
                                    torch.ones(1, device=DEV), amax))
    assert amax.item() == 0


@pytest.mark.parametrize("cols", [1, 7, 9, 133, 513, 1001, 4101, 12289, 17001])
@pytest.mark.parametrize("xt", [BF, F32])
def test_in_place(F, cols, xt):
    rows = 700 if cols < 5000 else 300
    g = torch.Generator(device=DEV).manual_seed(cols)
    new = lambda dt: torch.randn(rows, cols, generator=g, device=DEV).to(dt)  # noqa: E731
    x, d, dy, res, w = new(xt), new(BF), new(BF), new(xt), torch.rand(cols, device=DEV)
    h, y, r = torch.empty_like(x), empty(BF, rows, cols), empty(F32, rows)
    F.fp8_rmsnorm_fwd(x, d, w, 1e-5, h, y, r)
    x2, d2, y2 = x.clone(), d.clone(), torch.empty_like(y)
    F.fp8_rmsnorm_fwd(x2, d2, w, 1e-5, x2, d2, r)            # h over x, y over delta
    assert torch.equal(x2, h) and torch.equal(d2, y)
    if xt == BF:
        x2, d2 = x.clone(), d.clone()
        F.fp8_rmsnorm_fwd(x2, d2, w, 1e-5, d2, x2, r)        # and the other way round
        assert torch.equal(d2, h) and torch.equal(x2, y)
    dx, dg = torch.empty_like(x), empty(F32, cols)
    F.fp8_rmsnorm_bwd(dy, h, r, w, res, dx, dg)
    for over in ("h", "res") + (("dy",) if xt == BF else ()):
        t = {"h": h.clone(), "res": res.clone(), "dy": dy.clone()}
        dg2 = torch.empty_like(dg)
        F.fp8_rmsnorm_bwd(t["dy"], t["h"], r, w, t["res"], t[over], dg2)
        assert torch.equal(t[over], dx) and torch.equal(dg, dg2), over


def test_streams_and_graph(F):
    """On another stream, and captured with its workspaces: every replay gives
    the eager bits, with eager work between the replays."""
    rows, cols = 515, 1500
    x, d, gamma = (dev(t) for t in case(rows, cols, F32, F32, True))
    dy = normal(5, rows, cols).to(DEV)
    q, s = empty(torch.uint8, rows, cols), torch.full((1,), 16.0, device=DEV)

    def outputs():
        return dict(h=empty(F32, rows, cols), y=empty(BF, rows, cols), r=empty(F32, rows),
                    q=torch.zeros_like(q), amax=empty(F32, 1), dx=empty(F32, rows, cols),
                    dg=empty(F32, cols), ws=F.workspace(), wb=F.rmsnorm_workspace(rows, cols))

    def both(o, stream=None):
        F.fp8_rmsnorm_fwd(x, d, gamma, 1e-5, o["h"], o["y"], o["r"],
                          yq=F.cast_out(o["q"], 0, TENSOR, None, s, o["amax"]),
                          workspace=o["ws"], stream=stream)
        F.fp8_rmsnorm_bwd(dy, o["h"], o["r"], gamma, x, o["dx"], o["dg"], workspace=o["wb"],
                          stream=stream)
    names = ("h", "y", "r", "q", "amax", "dx", "dg")
    want = outputs()
    both(want)
    side, other = torch.cuda.Stream(), outputs()
    torch.cuda.synchronize()
    both(other, side)
    side.synchronize()
    assert all(torch.equal(want[n], other[n]) for n in names)
    got, graph = outputs(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        both(got)
    for i in range(4):
        for n in names:
            got[n].fill_(i)
        graph.replay()
        both(other)
        torch.cuda.synchronize()
        assert all(torch.equal(want[n], got[n]) for n in names), i


def test_more_than_2_31_elements(F):
    rows, cols = (1 << 31) // 8192 + 3, 8192
    x = torch.randn(rows, cols, device=DEV, dtype=BF)
    gamma = torch.ones(cols, device=DEV)
    y, r = torch.empty_like(x), empty(F32, rows)
    F.fp8_rmsnorm_fwd(x, None, gamma, 1e-5, None, y, r)
    dx, dg = torch.empty_like(x), empty(F32, cols)
    F.fp8_rmsnorm_bwd(y, x, r, gamma, x, dx, dg)
    tail = x[-9:].cpu().double()
    rstd, xhat, want = M.rms_fwd(tail, torch.ones(cols, dtype=torch.float64), 1e-5)
    R.check_bf16(y[-9:], want, M.rms_fwd_bounds(rstd, xhat, want)[2], "y")
    dy, rr = y[-9:].cpu().double(), r[-9:].cpu().double()
    xh = tail * rr[:, None]
    one = torch.ones(cols, dtype=torch.float64)
    wx, _ = M.rms_bwd(dy, xh, rr, one, tail)
    R.check_bf16(dx[-9:], wx, M.rms_bwd_bounds(dy, xh, M.U * xh.abs(), rr, one, tail)[0], "dx")
