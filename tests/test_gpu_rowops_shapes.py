"""The row operators where the kernels' division of the work changes: widths
at and around each number of slots per thread and of threads per row, more
rows than the chip holds at once, rows barely longer than a slot, and the
1x128 scales of every mantissa.  Bounds as in test_gpu_rowops."""
import numpy as np
import pytest
import torch

from tests import rowop_reference as R
from tests.gpu_helpers import DEV
from tests.test_gpu_rowops import (BLOCK, F, MX, NONE, TENSOR, empty, ln_case,  # noqa: F401
                                   make_cast, normal)

pytestmark = pytest.mark.gpu

# (rows, cols): several rows for every workgroup; few rows, one slot a thread;
# the widths where threads per row and slots per thread change
SHAPES = [(9000, 40), (5000, 700), (9001, 1025), (2500, 2049), (257, 4095), (256, 4096),
          (1500, 6144), (600, 6152), (700, 8193), (700, 12288), (300, 12296), (600, 16384),
          (520, 16392), (260, 20000)]


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt,scaling", [(torch.bfloat16, MX), (torch.float32, TENSOR)])
def test_layernorm_many_rows(F, rows, cols, xt, scaling):  # noqa: F811
    x, gamma, beta = ln_case(rows, cols, rows + cols, xt, torch.float32)
    pick = torch.arange(0, rows, max(1, rows // 40))
    pick = torch.cat([pick, torch.tensor([rows - 1])])
    xd = [x[pick].double(), gamma.double(), beta.double()]
    mean, rstd, xhat, y = R.ln_fwd(*xd, 1e-5)
    tm, tr, th, ty = R.ln_fwd_bounds(*xd, mean, rstd, xhat)
    yo, mo, ro = (empty(torch.bfloat16, rows, cols), empty(torch.float32, rows),
                  empty(torch.float32, rows))
    scale, amax = torch.full((1,), 32.0, device=DEV), empty(torch.float32, 1)
    q, s, yq = make_cast(F, rows, cols, scaling, 0, scale=scale, amax=amax)
    cq, cs, ck = make_cast(F, rows, cols, BLOCK)
    F.fp8_layernorm_fwd(x.to(DEV), gamma.to(DEV), beta.to(DEV), 1e-5, yo, mo, ro, yq=yq, xhat=ck)
    at = pick.to(DEV)
    R.check_close(mo[at], mean, tm + R.U * mean.abs(), "mean")
    R.check_close(ro[at], rstd, tr, "rstd")
    R.check_bf16(yo[at], y, ty, "y")
    R.check_cast(cq[at], cs[at], xhat, th, 0, BLOCK, "xhat")
    R.check_cast(q[at], None if s is None else s[at], y, ty, 0, scaling, "yq", scale=32.0)
    # every row: outputs were written and are finite
    assert torch.isfinite(yo).all() and torch.isfinite(mo).all() and torch.isfinite(ro).all()
    assert torch.isfinite(cs).all()
    if scaling == TENSOR:
        # BF16 rounding is monotonic: the largest output is the amax's
        assert amax.bfloat16().item() == yo.abs().max().item()


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("xt,held", [(torch.bfloat16, True), (torch.bfloat16, False),
                                     (torch.float32, False)])
def test_layernorm_bwd_many_rows(F, rows, cols, xt, held):  # noqa: F811
    x, gamma, beta = ln_case(rows, cols, 3 + rows + cols, xt, torch.bfloat16)
    dy = normal(rows * cols, rows, cols)
    mo, ro = empty(torch.float32, rows), empty(torch.float32, rows)
    cq, cs, ck = make_cast(F, rows, cols, BLOCK, 1)
    F.fp8_layernorm_fwd(x.to(DEV), gamma.to(DEV), beta.to(DEV), 1e-5, None, mo, ro, xhat=ck)
    dx = empty(xt, rows, cols)
    dg, db = empty(torch.float32, cols), empty(torch.float32, cols)
    if held:
        F.fp8_layernorm_bwd(dy.to(DEV), None, None, ro, gamma.to(DEV), dx, dg, db,
                            xhat=F.operand(cq, F.E5M2, F.SCALE_BLOCK_1x128, cs))
        xhat = R.held_values(cq, cs, 1)
        t_xhat = R.U * xhat.abs()
    else:
        F.fp8_layernorm_bwd(dy.to(DEV), x.to(DEV), mo, ro, gamma.to(DEV), dx, dg, db)
        m, r = mo.cpu().double(), ro.cpu().double()
        xhat = (x.double() - m[:, None]) * r[:, None]
        t_xhat = 3 * R.U * xhat.abs()
    r, g = ro.cpu().double(), gamma.double()
    wx, wg, wb = R.ln_bwd(dy.double(), xhat, r, g)
    tx, tg, tb = R.ln_bwd_bounds(dy.double(), xhat, t_xhat, r, g)
    if xt == torch.bfloat16:
        R.check_bf16(dx, wx, tx, "dx")
    else:
        R.check_close(dx, wx, tx + R.U * wx.abs(), "dx")
    R.check_close(dg, wg, tg, "dgamma")
    R.check_close(db, wb, tb, "dbeta")


def test_scales_of_every_mantissa(F):  # noqa: F811
    """1x128 scales are FP32 quotients rounded to nearest: scale_inv =
    1 / (448 / amax) for every amax in [1, 2).  A row of zeros makes y = beta,
    whose tiles hold one value each."""
    tiles, calls = 256, 1 << 15
    cols = tiles * 128
    values = np.arange(1 << 23, dtype=np.uint32) + np.uint32(0x3f800000)
    amax = torch.from_numpy(values.view(np.float32)).to(DEV).view(calls, tiles)
    x = torch.zeros((1, cols), device=DEV)
    gamma, beta = torch.ones(cols, device=DEV), torch.zeros(cols, device=DEV)
    spots = beta.view(tiles, 128)[:, 77]
    mo, ro = empty(torch.float32, 1), empty(torch.float32, 1)
    q = empty(torch.uint8, 1, cols)
    s = empty(torch.float32, calls, tiles)
    outs = [F.cast_out(q, F.E4M3, F.SCALE_BLOCK_1x128, s[i]) for i in range(calls)]
    for i in range(calls):
        spots.copy_(amax[i])
        F.fp8_layernorm_fwd(x, gamma, beta, 1e-5, None, mo, ro, yq=outs[i])
    a = values.view(np.float32)
    want = np.float32(1) / (np.float32(448) / a)
    assert (s.cpu().numpy().reshape(-1) == want).all()
    assert (q.view(tiles, 128)[:, 77] == 0x7e).all()      # the largest value is +-448


@pytest.mark.parametrize("exponent", [-126, -100, -81, -80, -79, 0, 99, 100, 101, 127])
@pytest.mark.parametrize("fmt,top", [(0, 448.0), (1, 57344.0)])
def test_scales_far_out(F, exponent, fmt, top):  # noqa: F811
    """The scale rule at FP32's ends, where the general division is used."""
    cols = 128 * 40
    g = np.random.default_rng(exponent + 200)
    a = np.ldexp(1 + g.random(40), exponent).astype(np.float32)
    a[7], a[8] = 0.0, np.float32(np.ldexp(1.0, exponent))
    beta = torch.zeros(40, 128)
    beta[:, 5] = torch.from_numpy(a)
    q, s, yq = make_cast(F, 1, cols, BLOCK, fmt)
    F.fp8_layernorm_fwd(torch.zeros((1, cols), device=DEV), torch.ones(cols, device=DEV),
                        beta.view(-1).to(DEV), 1e-5, None, empty(torch.float32, 1),
                        empty(torch.float32, 1), yq=yq)
    with np.errstate(all="ignore"):
        scale = np.where(a > 0, np.minimum(np.float32(top) / a, np.finfo(np.float32).max),
                         np.float32(1)).astype(np.float32)
        want = np.float32(1) / scale
    assert (s.cpu().numpy().reshape(-1) == want).all()


# rows of one slot and a little more, in every operator that reads rows
@pytest.mark.parametrize("cols", [1, 2, 7, 8, 9, 11, 15, 16, 23, 31])
def test_short_rows(F, cols):  # noqa: F811
    rows = 37
    h = normal(cols, rows, 2 * cols)
    dy = normal(cols + 1, rows, cols)
    hd, dd = h.double(), dy.double()
    a, u = hd[:, :cols], hd[:, cols:]
    p, d = R.act_parts(2, a)
    y, dh = empty(torch.bfloat16, rows, cols), empty(torch.bfloat16, rows, 2 * cols)
    cq, cs, ck = make_cast(F, rows, cols, BLOCK, halves=2)
    F.fp8_act_fwd(h.to(DEV), F.ACT_SILU, True, y, ckpt=ck)
    want = a * p * u
    R.check_bf16(y, want, 16 * R.U * want.abs(), "y")
    F.fp8_act_bwd(dy.to(DEV), h.to(DEV), F.ACT_SILU, True, dh)
    want = torch.cat([dd * u * d, dd * a * p], 1)
    # act' = p (1 + a (1 - p)) may cancel: count its terms
    slack = torch.cat([dd * u * p * (1 + a.abs() * (1 - p)), dd * a * p], 1).abs()
    R.check_bf16(dh, want, 16 * R.U * slack, "dh")
    # a checkpoint keeps each half's rows apart
    held = R.held_values(cq.view(-1, cols), cs, 0).reshape(rows, 2 * cols)
    x2 = h.to(DEV).view(-1, cols)
    q2, s2, c2 = make_cast(F, rows * 2, cols, BLOCK)
    back = empty(torch.bfloat16, rows * 2, cols)
    F.fp8_checkpoint_save(x2, c2)
    F.fp8_checkpoint_load(F.operand(q2, F.E4M3, F.SCALE_BLOCK_1x128, s2), rows * 2, cols, back)
    assert torch.equal(q2.view(-1), cq.view(-1)) and torch.equal(s2.view(-1), cs.view(-1))
    R.check_bf16(back.view(rows, 2 * cols), held, R.U * held.abs(), "loaded")


# dispatch with 1, 2 and 4 slots a lane, several shares of a row, small and
# large batches' padding
@pytest.mark.parametrize("tokens,k,experts,cols,pad", [
    (4200, 2, 8, 600, 16), (2100, 1, 4, 1100, 128), (1400, 3, 8, 2200, 1), (3, 2, 8, 5000, 16),
    (900, 2, 64, 4100, 128)])
def test_dispatch_shares(F, tokens, k, experts, cols, pad):  # noqa: F811
    g = torch.Generator().manual_seed(tokens)
    expert = torch.randint(-1, experts, (tokens, k), generator=g, dtype=torch.int32).to(DEV)
    x = normal(cols, tokens, cols).to(DEV)
    n = tokens * k
    r = F.moe_rows(n, experts, pad)
    off, cnt = empty(torch.int32, experts + 1), empty(torch.int32, experts)
    pos, src = empty(torch.int32, tokens, k), empty(torch.int32, r)
    F.fp8_moe_sort(expert, experts, pad, off, cnt, pos, src)
    xs = torch.full((r, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    q, s, xq = make_cast(F, r, cols, BLOCK)
    F.fp8_moe_dispatch(x, pos, src, off, xs, xq=xq)
    end = off[-1].item()
    real = src >= 0
    want = torch.where(real[:, None], x[torch.where(real, src // k, 0).long()], 0.0)
    assert torch.equal(xs[:end], want[:end].bfloat16())
    assert (xs[end:] == 7.0).all()
    q2, s2, c2 = make_cast(F, end, cols, BLOCK)
    F.fp8_checkpoint_save(xs[:end].contiguous(), c2)
    assert torch.equal(q[:end], q2) and torch.equal(s[:end], s2)


def test_more_rows_than_one_grid(F):  # noqa: F811
    """Rows beyond what one launch's threads reach: the kernels loop."""
    tokens, cols = (1 << 24) + 21, 8
    x = torch.arange(tokens * cols, dtype=torch.int32, device=DEV).view(tokens, cols)
    x = (x % 251 - 125).to(torch.bfloat16)
    pos = torch.arange(tokens - 1, -1, -1, dtype=torch.int32, device=DEV).view(tokens, 1)
    off = torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    xs, y, dys = (empty(torch.bfloat16, tokens, cols) for _ in range(3))
    F.fp8_moe_dispatch(x, pos, pos.view(-1), off, xs)
    assert torch.equal(xs, x.flip(0))
    F.fp8_moe_combine(xs, pos, None, y)
    assert torch.equal(y, x)
    w, dw = torch.full((tokens, 1), 2.0, device=DEV), empty(torch.float32, tokens, 1)
    F.fp8_moe_combine_bwd(x, xs, w, pos, pos.view(-1), off, dys, dw)
    assert torch.equal(dys, 2 * xs)
    assert torch.equal(dw[:, 0], (x.float() ** 2).sum(1))     # whole numbers below 2^24
    # padding rows: none of 2^26 + 37 rows is a token's
    rows = (1 << 26) + 37
    src = torch.full((rows,), -1, dtype=torch.int32, device=DEV)
    off = torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    none = torch.full((1, 1), -1, dtype=torch.int32, device=DEV)
    xs = torch.ones((rows, 1), dtype=torch.bfloat16, device=DEV)
    F.fp8_moe_dispatch(torch.ones_like(xs[:1]), none, src, off, xs)
    assert not xs.any()
    # one tile a row
    v = torch.arange(rows, dtype=torch.int32, device=DEV).view(rows, 1)
    v = (v % 97 - 48).to(torch.bfloat16)
    q, s, ck = make_cast(F, rows, 1, BLOCK)
    F.fp8_checkpoint_save(v, ck)
    F.fp8_checkpoint_load(F.operand(q, F.E4M3, F.SCALE_BLOCK_1x128, s), rows, 1, xs)
    assert torch.equal(xs, v)                                 # +-448 / (448 / |v|)
