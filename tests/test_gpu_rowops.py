"""GPU parity of the row operators (layer norm, activations, 8-bit
checkpoints, expert sorting) with their formulas in 64 bits, under the bounds
of rowop_reference; casts of BF16 inputs equal the oracle's bytes and scales
bit for bit."""
import numpy as np
import pytest
import torch

from tests import rowop_reference as R
from tests.gpu_helpers import DEV, bits16, bytes8

pytestmark = pytest.mark.gpu

NONE, TENSOR, BLOCK, MX = -1, 0, 1, 3


@pytest.fixture(scope="module")
def F():
    from scaled_fp8_gemm_amd import fp8sg
    fp8sg.lib()
    return fp8sg


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def empty(dtype, *shape):
    """Device memory that holds no plausible result."""
    if dtype.is_floating_point:
        return torch.full(shape, float("nan"), dtype=dtype, device=DEV)
    return torch.full(shape, 0x7f, dtype=dtype, device=DEV)


def make_cast(F, rows, cols, scaling, fmt=0, halves=1, scale=None, amax=None):
    q = empty(torch.uint8, rows, cols * halves)
    s = None
    if scaling == BLOCK:
        s = empty(torch.float32, rows * halves, -(-cols // 128))
    elif scaling == MX:
        s = empty(torch.uint8, rows * halves, -(-cols // 32))
    return q, s, F.cast_out(q, fmt, scaling, s, scale, amax)


def oracle_tiles(orc, x, fmt=0):
    """The oracle's 1x128 cast of BF16 rows of any length: rows filled up with
    zeros, which change no tile's maximum."""
    r, c = x.shape
    n = -(-c // 128) * 128
    b = np.zeros((r, n), np.uint16)
    b[:, :c] = bits16(x)
    q, s = orc.quantize_block(b, fmt, 1, 128)
    return q[:, :c], s


def oracle_mx(orc, x, fmt=0):
    r, c = x.shape
    b = np.zeros((r, -(-c // 32) * 32), np.uint16)
    b[:, :c] = bits16(x)
    q, e = orc.quantize_mx(b, fmt)
    return q[:, :c], e


# ------------------------------------------------------------ layer norm
# widths that end inside a slot, a tile, a wave's share, at and across each
# number of slots per thread, up to the limit
LN_SHAPES = [(1, 1), (3, 7), (5, 8), (4, 127), (9, 129), (6, 512), (5, 513), (7, 1003), (3, 1024),
             (2, 1025), (4, 2048), (3, 2057), (3, 4096), (2, 8195), (2, 12288), (1, 16384),
             (2, 32768)]


def ln_case(rows, cols, seed, xt, wt):
    x = normal(seed, rows, cols, dtype=torch.float32) + 0.5 * normal(seed + 1, rows, 1,
                                                                     dtype=torch.float32)
    return (x.to(xt), (1 + 0.2 * normal(seed + 2, cols, dtype=torch.float32)).to(wt),
            normal(seed + 3, cols, dtype=torch.float32, scale=0.1).to(wt))


@pytest.mark.parametrize("shape", LN_SHAPES)
@pytest.mark.parametrize("xt,wt,scaling,fmt", [
    (torch.bfloat16, torch.float32, MX, 0), (torch.bfloat16, torch.bfloat16, BLOCK, 1),
    (torch.float32, torch.float32, TENSOR, 0), (torch.float32, torch.bfloat16, NONE, 0)])
def test_layernorm_fwd(F, shape, xt, wt, scaling, fmt):
    rows, cols = shape
    x, gamma, beta = ln_case(rows, cols, rows + cols, xt, wt)
    xd = [v.double() for v in (x, gamma, beta)]
    mean, rstd, xhat, y = R.ln_fwd(*xd, 1e-5)
    tm, tr, th, ty = R.ln_fwd_bounds(*xd, mean, rstd, xhat)
    yo, mo, ro = empty(torch.bfloat16, rows, cols), empty(torch.float32, rows), empty(torch.float32,
                                                                                   rows)
    scale, amax = torch.full((1,), 32.0, device=DEV), empty(torch.float32, 1)
    q = s = yq = None
    if scaling != NONE:
        q, s, yq = make_cast(F, rows, cols, scaling, fmt, scale=scale, amax=amax)
    cq, cs, ck = make_cast(F, rows, cols, BLOCK)
    F.fp8_layernorm_fwd(x.to(DEV), gamma.to(DEV), beta.to(DEV), 1e-5, yo, mo, ro, yq=yq, xhat=ck)
    R.check_close(mo, mean, tm + R.U * mean.abs(), "mean")
    R.check_close(ro, rstd, tr, "rstd")
    R.check_bf16(yo, y, ty, "y")
    R.check_cast(cq, cs, xhat, th, 0, BLOCK, "xhat")
    if scaling != NONE:
        R.check_cast(q, s, y, ty, fmt, scaling, "yq", scale=32.0)
    if scaling == TENSOR:
        R.check_close(amax, y.abs().max(), ty.max(), "amax")


@pytest.mark.parametrize("shape", LN_SHAPES + [(300, 264), (1100, 200), (700, 1400)])
@pytest.mark.parametrize("xt,wt,held", [
    (torch.bfloat16, torch.float32, True), (torch.float32, torch.bfloat16, True),
    (torch.bfloat16, torch.bfloat16, False), (torch.float32, torch.float32, False)])
def test_layernorm_bwd(F, shape, xt, wt, held):
    rows, cols = shape
    x, gamma, beta = ln_case(rows, cols, 7 + rows + cols, xt, wt)
    dy = normal(rows * cols, rows, cols)
    # one pass makes what the other takes
    mo, ro = empty(torch.float32, rows), empty(torch.float32, rows)
    cq, cs, ck = make_cast(F, rows, cols, BLOCK)
    F.fp8_layernorm_fwd(x.to(DEV), gamma.to(DEV), beta.to(DEV), 1e-5, None, mo, ro, xhat=ck)
    dx = empty(xt, rows, cols)
    dg, db = empty(torch.float32, cols), empty(torch.float32, cols)
    args = (dx, dg, db)
    if held:
        F.fp8_layernorm_bwd(dy.to(DEV), None, None, ro, gamma.to(DEV), *args,
                            xhat=F.operand(cq, F.E4M3, F.SCALE_BLOCK_1x128, cs))
        xhat = R.held_values(cq, cs, 0)
        t_xhat = R.U * xhat.abs()
    else:
        F.fp8_layernorm_bwd(dy.to(DEV), x.to(DEV), mo, ro, gamma.to(DEV), *args)
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


def test_layernorm_without_rows(F):
    x = torch.empty((0, 40), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(40, device=DEV)
    e = torch.empty(0, device=DEV)
    amax, scale = empty(torch.float32, 1), torch.ones(1, device=DEV)
    q = torch.empty((0, 40), dtype=torch.uint8, device=DEV)
    F.fp8_layernorm_fwd(x, w, w, 1e-5, x, e, e, yq=F.cast_out(q, 0, TENSOR, None, scale, amax))
    assert amax.item() == 0
    dg, db = empty(torch.float32, 40), empty(torch.float32, 40)
    F.fp8_layernorm_bwd(x, x, e, e, w, x, dg, db)
    assert not dg.any() and not db.any()


def test_layernorm_special_rows(F):
    """NaN and infinities stay in their rows; a row of one value has xhat 0."""
    rows, cols = 6, 1000
    x, gamma, beta = ln_case(rows, cols, 3, torch.float32, torch.float32)
    x[1, 500] = float("nan")
    x[2, 999] = float("inf")
    x[4] = 3.25
    y, mo, ro = (empty(torch.bfloat16, rows, cols), empty(torch.float32, rows),
                 empty(torch.float32, rows))
    q, s, yq = make_cast(F, rows, cols, MX)
    cq, cs, ck = make_cast(F, rows, cols, BLOCK)
    F.fp8_layernorm_fwd(x.to(DEV), gamma.to(DEV), beta.to(DEV), 1e-5, y, mo, ro, yq=yq, xhat=ck)
    y = y.float().cpu()
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    assert (bytes8(q)[1:3] == 0xff).all() and (bytes8(s)[1:3] == 0xff).all()
    assert (bytes8(cq)[1] == 0xff).all() and (cs.cpu()[1] == 1).all()
    assert torch.isfinite(y[[0, 3, 4, 5]]).all()
    assert not bytes8(cq)[4].any() and (cs.cpu()[4] == 1).all()
    assert torch.equal(y[4], beta.bfloat16().float())


# ------------------------------------------------------------ activations
ACT_SHAPES = [(1, 1), (3, 9), (5, 64), (7, 127), (4, 128), (6, 130), (33, 1001), (17, 1408),
              (64, 2056), (2, 16384)]


@pytest.mark.parametrize("shape", ACT_SHAPES)
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("gated,scaling,fmt", [(False, BLOCK, 1), (True, BLOCK, 0),
                                               (False, MX, 0), (True, MX, 1), (False, TENSOR, 0),
                                               (True, TENSOR, 1), (True, NONE, 0)])
def test_act_fwd(F, orc, shape, act, gated, scaling, fmt):
    rows, cols = shape
    w = 2 if gated else 1
    h = normal(rows + cols + act, rows, cols * w, scale=2.5)
    hd = h.double()
    a = hd[:, :cols]
    p, _ = R.act_parts(act, a)
    rel, _ = R.act_bounds(act, a)
    y = a * p
    tol = y.abs() * (rel + 3 * R.U)
    if gated:
        y, tol = y * hd[:, cols:], tol * hd[:, cols:].abs() * (1 + 2 * R.U)
        tol = tol + R.U * y.abs()
    yo = empty(torch.bfloat16, rows, cols)
    scale, amax = torch.full((1,), 16.0, device=DEV), empty(torch.float32, 1)
    q = s = yq = None
    if scaling != NONE:
        q, s, yq = make_cast(F, rows, cols, scaling, fmt, scale=scale, amax=amax)
    cq, cs, ck = make_cast(F, rows, cols, BLOCK, fmt, halves=w)
    F.fp8_act_fwd(h.to(DEV), act, gated, yo, yq=yq, ckpt=ck)
    R.check_bf16(yo, y, tol, "y")
    if scaling != NONE:
        R.check_cast(q, s, y, tol, fmt, scaling, "yq", scale=16.0)
    if scaling == TENSOR:
        R.check_close(amax, y.abs().max(), tol.max() + R.U * y.abs().max(), "amax")
    wq, ws = oracle_tiles(orc, h.view(rows * w, cols), fmt)
    assert np.array_equal(bytes8(cq).reshape(rows * w, cols), wq)
    assert np.array_equal(cs.cpu().numpy(), ws)


@pytest.mark.parametrize("shape", ACT_SHAPES)
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("held,fmt", [(False, 0), (True, 0), (True, 1)])
def test_act_bwd(F, shape, act, gated, held, fmt):
    rows, cols = shape
    w = 2 if gated else 1
    h = normal(rows + cols + act, rows, cols * w, scale=2.5)
    dy = normal(rows * cols, rows, cols)
    dh, yo = empty(torch.bfloat16, rows, cols * w), empty(torch.bfloat16, rows, cols)
    t_h = torch.zeros(1, dtype=torch.float64)
    if held:
        cq, cs, ck = make_cast(F, rows * w, cols, BLOCK, fmt)
        F.fp8_checkpoint_save(h.view(rows * w, cols).to(DEV), ck)
        F.fp8_act_bwd(dy.to(DEV), F.operand(cq, fmt, F.SCALE_BLOCK_1x128, cs), act, gated, dh, y=yo)
        hd = R.held_values(cq, cs, fmt).reshape(rows, cols * w)
        t_h = R.U                        # of the value: one product in FP32
    else:
        F.fp8_act_bwd(dy.to(DEV), h.to(DEV), act, gated, dh, y=yo)
        hd = h.double()
    a, g = hd[:, :cols], dy.double()
    p, d = R.act_parts(act, a)
    rel, td = R.act_bounds(act, a)
    # a rounding of h moves the slope by at most 3 |h| of its step
    td = td + 3 * t_h * a.abs()
    y = a * p
    ty = y.abs() * (rel + 4 * R.U) + 3 * t_h * a.abs()
    if gated:
        u = hd[:, cols:]
        R.check_bf16(dh[:, :cols].contiguous(), g * u * d,
                     (g * u).abs() * (td + 4 * R.U * d.abs()), "da")
        R.check_bf16(dh[:, cols:].contiguous(), g * y, g.abs() * (ty + 2 * R.U * y.abs()), "du")
        R.check_bf16(yo, y * u, u.abs() * (ty + 4 * R.U * y.abs()), "y")
    else:
        R.check_bf16(dh, g * d, g.abs() * (td + 2 * R.U * d.abs()), "dh")
        R.check_bf16(yo, y, ty, "y")


@pytest.mark.parametrize("act", [0, 1, 2])
def test_act_far_out(F, act):
    """Large finite inputs: act(h) is h or 0, its slope 1 or 0, no NaN; NaN
    stays where it is."""
    h = torch.tensor([[50.0, -50.0, 1e4, -1e4, 1e18, -1e18, 3e38, -3e38, 0.0, -0.0, float("nan"),
                       1.0]]).bfloat16()
    dy = torch.ones_like(h)
    y, dh, y2 = (empty(torch.bfloat16, 1, 12) for _ in range(3))
    F.fp8_act_fwd(h.to(DEV), act, False, y)
    F.fp8_act_bwd(dy.to(DEV), h.to(DEV), act, False, dh, y=y2)
    hv, yv, dv = h.float()[0], y.float().cpu()[0], dh.float().cpu()[0]
    for i in range(0, 8, 2):
        assert yv[i] == hv[i] and dv[i] == 1, (i, yv[i], dv[i])
        # silu(-50) = -50 e^-50 is a number yet
        p, d = R.act_parts(act, hv[i + 1].double())
        want_y, want_d = (hv[i + 1] * p).item(), d.item()
        if i:
            assert want_y == 0
        assert abs(yv[i + 1] - want_y) <= 0.01 * abs(want_y), (i, yv[i + 1])
        assert abs(dv[i + 1] - want_d) <= 0.01 * abs(want_d), (i, dv[i + 1])
    assert yv[8] == 0 and yv[9] == 0 and (dv[8:10] == 0.5).all()
    assert torch.isnan(yv[10]) and torch.isnan(dv[10])
    assert torch.equal(y.view(torch.int16), y2.view(torch.int16))


# ------------------------------------------------------------ checkpoints
@pytest.mark.parametrize("shape", ACT_SHAPES + [(0, 5), (5, 0), (1000, 384)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_checkpoint(F, orc, shape, fmt):
    rows, cols = shape
    x = normal(rows + 3 * cols, rows, cols, scale=3.0)
    if rows * cols > 64:
        flat = x.view(-1)
        flat[::17] *= 1e-3
        flat[5], flat[rows * cols // 2] = float("inf"), float("nan")
        flat[-3:] = torch.tensor([3.3e38, 1e-40, 0.0]).bfloat16()
    q, s, ck = make_cast(F, rows, cols, BLOCK, fmt)
    F.fp8_checkpoint_save(x.to(DEV), ck)
    y = empty(torch.bfloat16, rows, cols)
    F.fp8_checkpoint_load(F.operand(q, fmt, F.SCALE_BLOCK_1x128, s), rows, cols, y)
    if not rows * cols:
        return
    wq, ws = oracle_tiles(orc, x, fmt)
    assert np.array_equal(bytes8(q), wq)
    assert np.array_equal(s.cpu().numpy().view(np.uint32), ws.view(np.uint32))
    v = R.tiles(q.cpu().view(R.FP8[fmt]).float(), 128) * s.cpu()[:, :, None]
    v = v.view(rows, -1)[:, :cols].bfloat16()
    g = y.cpu()
    assert torch.equal(torch.isnan(g), torch.isnan(v))
    assert torch.equal(torch.nan_to_num(g), torch.nan_to_num(v))


# ------------------------------------------------------------ expert sorting
def choices(seed, tokens, k, experts, drop=0.1):
    g = torch.Generator().manual_seed(seed)
    e = torch.randint(0, experts, (tokens, k), generator=g, dtype=torch.int32)
    out = torch.rand((tokens, k), generator=g) < drop
    e[out] = -1
    if e.numel() > 3:
        e.view(-1)[0], e.view(-1)[1] = experts, -2 ** 31
        e.view(-1)[2] = 2 ** 31 - 1
    return e


def run_sort(F, e, experts, pad, extra=0):
    rows = F.moe_rows(e.numel(), experts, pad) + extra
    out = [empty(torch.int32, experts + 1), empty(torch.int32, experts),
           empty(torch.int32, *e.shape), empty(torch.int32, rows)]
    F.fp8_moe_sort(e.to(DEV), experts, pad, *out)
    return rows, out


@pytest.mark.parametrize("tokens,k,experts,pad", [
    (0, 2, 4, 16), (1, 1, 1, 1), (1, 8, 8, 128), (16, 2, 8, 16), (63, 1, 2, 3), (64, 3, 40, 1),
    (1024, 1, 7, 5), (1025, 2, 64, 128), (5000, 6, 128, 16), (9000, 10, 1024, 2),
    (40000, 2, 1000, 128), (66000, 1, 8, 1), (1100000, 1, 16, 128)])
def test_moe_sort(F, tokens, k, experts, pad):
    e = choices(tokens + k, tokens, k, experts)
    rows, got = run_sort(F, e, experts, pad, extra=tokens % 5)
    for name, g, w in zip(("offsets", "counts", "pos", "src"), got,
                          R.sort_choices(e, experts, pad, rows)):
        assert torch.equal(g.cpu(), w), name


@pytest.mark.parametrize("which", ["one", "dropped", "last"])
def test_moe_sort_uneven(F, which):
    e = torch.full((3000, 2), {"one": 3, "dropped": -1, "last": 11}[which], dtype=torch.int32)
    rows, got = run_sort(F, e, 12, 16)
    for g, w in zip(got, R.sort_choices(e, 12, 16, rows)):
        assert torch.equal(g.cpu(), w)


MOE = [(0, 2, 4, 64, 16), (1, 1, 1, 1, 1), (5, 2, 8, 7, 16), (16, 2, 8, 4096, 16),
       (77, 3, 5, 1001, 128), (130, 6, 64, 130, 1), (64, 10, 16, 513, 16), (2500, 8, 40, 72, 128),
       (2100, 1, 4, 1030, 16), (300, 4, 8, 8192, 128), (90, 5, 8, 128, 16), (90, 7, 8, 136, 16)]


def moe_case(F, tokens, k, experts, cols, pad):
    e = choices(tokens + cols, tokens, k, experts)
    if tokens > 4:
        e[3] = -1                                   # a token with nothing
    rows = F.moe_rows(e.numel(), experts, pad) + 3
    offsets, counts, pos, src = R.sort_choices(e, experts, pad, rows)
    return rows, offsets, pos, src, [v.to(DEV) for v in (pos, src, offsets)]


@pytest.mark.parametrize("tokens,k,experts,cols,pad", MOE)
@pytest.mark.parametrize("scaling", [NONE, TENSOR, BLOCK, MX])
def test_moe_dispatch(F, orc, tokens, k, experts, cols, pad, scaling):
    rows, offsets, pos, src, dev = moe_case(F, tokens, k, experts, cols, pad)
    x = normal(cols, tokens, cols)
    xs = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    scale = torch.full((1,), 50.0, device=DEV)
    q = s = xq = None
    if scaling != NONE:
        q, s, xq = make_cast(F, rows, cols, scaling, scale=scale)
    F.fp8_moe_dispatch(x.to(DEV), *dev, xs, xq=xq)
    want = torch.full((rows, cols), 7.0, dtype=torch.bfloat16)   # past the end: left alone
    end = int(offsets[-1])
    want[:end] = 0
    real = src >= 0
    want[real] = x[src[real].long() // k]
    assert torch.equal(xs.cpu(), want)
    if scaling == NONE or end == 0:
        return
    used = want[:end]
    if scaling == BLOCK:
        wq, ws = oracle_tiles(orc, used)
    elif scaling == MX:
        wq, ws = oracle_mx(orc, used)
    else:
        b = np.zeros((end, -(-cols // 16) * 16), np.uint16)
        b[:, :cols] = bits16(used)
        wq = orc.quantize_tensor(b, 0, np.float32(50.0))[0][:, :cols]
    assert np.array_equal(bytes8(q)[:end], wq)
    assert (bytes8(q)[end:] == 0x7f).all()
    if scaling in (BLOCK, MX):
        assert np.array_equal(s.cpu().numpy()[:end], ws)
        got = s.cpu()[end:]
        assert bool(torch.isnan(got).all() if scaling == BLOCK else (got == 0x7f).all())


@pytest.mark.parametrize("tokens,k,experts,cols,pad", MOE)
@pytest.mark.parametrize("weighted", [False, True])
def test_moe_combine(F, tokens, k, experts, cols, pad, weighted):
    rows, offsets, pos, src, dev = moe_case(F, tokens, k, experts, cols, pad)
    ys = normal(cols + 1, rows, cols)
    ys[src < 0] = float("nan")                      # rows that no choice names
    w = normal(3, tokens, k, dtype=torch.float32) if weighted else None
    if weighted:
        w[pos < 0] = float("nan")                   # weights of dropped choices
    y = empty(torch.bfloat16, tokens, cols)
    F.fp8_moe_combine(ys.to(DEV), dev[0], None if w is None else w.to(DEV), y)
    want, mag = (torch.zeros((tokens, cols), dtype=torch.float64) for _ in range(2))
    for j in range(k):
        ok = pos[:, j] >= 0
        t = ys[pos[ok, j].long()].double()
        if weighted:
            t = t * w[ok, j, None].double()
        want[ok] += t
        mag[ok] += t.abs()
    R.check_bf16(y, want, (k + 1) * R.U * mag, "y")


@pytest.mark.parametrize("tokens,k,experts,cols,pad", MOE)
def test_moe_combine_bwd(F, tokens, k, experts, cols, pad):
    rows, offsets, pos, src, dev = moe_case(F, tokens, k, experts, cols, pad)
    dy, ys = normal(cols, tokens, cols), normal(cols + 1, rows, cols)
    ys[src < 0] = float("nan")
    w = normal(3, tokens, k, dtype=torch.float32)
    w[pos < 0] = float("nan")
    dys = torch.full((rows, cols), 7.0, dtype=torch.bfloat16, device=DEV)
    dw = empty(torch.float32, tokens, k)
    F.fp8_moe_combine_bwd(dy.to(DEV), ys.to(DEV), w.to(DEV), *dev, dys, dw)
    want = torch.full((rows, cols), 7.0, dtype=torch.float64)
    want[:int(offsets[-1])] = 0
    ww, mag = (torch.zeros((tokens, k), dtype=torch.float64) for _ in range(2))
    for j in range(k):
        ok = pos[:, j] >= 0
        at = pos[ok, j].long()
        want[at] = w[ok, j, None].double() * dy[ok].double()
        ww[ok, j] = (dy[ok].double() * ys[at].double()).sum(1)
        mag[ok, j] = (dy[ok].double() * ys[at].double()).abs().sum(1)
    R.check_bf16(dys, want, R.U * want.abs(), "dys")
    # a lane's elements one after the other (at most an eighth wave's share of
    # the row), then the tree
    R.check_close(dw, ww, (cols / 64 + 32) * R.U * mag, "dweight")


def test_moe_takes_positions_out_of_range_as_dropped(F):
    x, ys = normal(1, 4, 64), normal(2, 10, 64)
    pos = torch.tensor([[0], [10], [2 ** 31 - 1], [-5]], dtype=torch.int32, device=DEV)
    src = torch.full((10,), -1, dtype=torch.int32, device=DEV)
    src[0] = 0
    off = torch.tensor([0, 1000], dtype=torch.int32, device=DEV)    # past the rows there are
    xs = empty(torch.bfloat16, 10, 64)
    F.fp8_moe_dispatch(x.to(DEV), pos, src, off, xs)
    assert torch.equal(xs.cpu()[0], x[0]) and not xs.cpu()[1:].any()
    y = empty(torch.bfloat16, 4, 64)
    F.fp8_moe_combine(ys.to(DEV), pos, None, y)
    assert torch.equal(y.cpu()[0], ys[0]) and not y.cpu()[1:].any()


# ------------------------------------------------------------ all of them
def _everything(F, t, ws):
    """Each call once, into t's outputs; x: [rows][cols], gated half of it."""
    F.fp8_layernorm_fwd(t["x"], t["g"], t["b"], 1e-5, t["y"], t["mean"], t["rstd"],
                        yq=F.cast_out(t["q0"], 0, TENSOR, None, t["scale"], t["amax"]),
                        xhat=F.cast_out(t["ck"], 0, BLOCK, t["ck_s"]), workspace=ws["amax"])
    F.fp8_layernorm_bwd(t["dy"], None, None, t["rstd"], t["g"], t["dx"], t["dg"], t["db"],
                        xhat=F.operand(t["ck"], 0, BLOCK, t["ck_s"]), workspace=ws["ln"])
    F.fp8_act_fwd(t["x"], F.ACT_SILU, True, t["a"],
                  yq=F.cast_out(t["q1"], 0, TENSOR, None, t["scale"], t["amax1"]),
                  workspace=ws["amax"])
    F.fp8_act_bwd(t["a"], t["x"], F.ACT_SILU, True, t["da"])
    F.fp8_moe_sort(t["e"], 8, 16, t["off"], t["cnt"], t["pos"], t["src"], workspace=ws["moe"])
    F.fp8_moe_dispatch(t["x"], t["pos"], t["src"], t["off"], t["xs"])
    F.fp8_moe_combine(t["xs"], t["pos"], t["w"], t["yc"])
    F.fp8_moe_combine_bwd(t["dy"], t["xs"], t["w"], t["pos"], t["src"], t["off"], t["dys"], t["dw"])


def _tensors(F, rows, cols, seed):
    bf, f, u, i = torch.bfloat16, torch.float32, torch.uint8, torch.int32
    r = F.moe_rows(rows * 2, 8, 16)
    z = lambda dt, *s: torch.zeros(s, dtype=dt, device=DEV)  # noqa: E731
    t = dict(x=normal(seed, rows, cols).to(DEV), dy=normal(seed + 1, rows, cols).to(DEV),
             g=normal(seed + 2, cols).to(DEV), b=normal(seed + 3, cols).to(DEV),
             e=choices(seed, rows, 2, 8).to(DEV),
             w=normal(seed + 4, rows, 2, dtype=f).to(DEV), scale=torch.full((1,), 4.0, device=DEV))
    outs = dict(y=z(bf, rows, cols), mean=z(f, rows), rstd=z(f, rows), q0=z(u, rows, cols),
                amax=z(f, 1), ck=z(u, rows, cols), ck_s=z(f, rows, -(-cols // 128)),
                dx=z(bf, rows, cols), dg=z(f, cols), db=z(f, cols), a=z(bf, rows, cols // 2),
                q1=z(u, rows, cols // 2), amax1=z(f, 1), da=z(bf, rows, cols), off=z(i, 9),
                cnt=z(i, 8), pos=z(i, rows, 2), src=z(i, r), xs=z(bf, r, cols),
                yc=z(bf, rows, cols), dys=z(bf, r, cols), dw=z(f, rows, 2))
    return t, outs


def test_row_operators_in_a_graph(F):
    rows, cols = 700, 1030
    ins, eager = _tensors(F, rows, cols, 5)
    ws = dict(amax=F.workspace(), ln=F.layernorm_workspace(rows, cols),
              moe=F.moe_workspace(rows * 2, 8))
    _everything(F, {**ins, **eager}, ws)
    torch.cuda.synchronize()
    _, cap = _tensors(F, rows, cols, 5)
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        _everything(F, {**ins, **cap}, ws)
    other_in, other = _tensors(F, 300, 264, 9)
    ows = dict(amax=F.workspace(), ln=F.layernorm_workspace(300, 264), moe=F.moe_workspace(600, 8))
    for rep in range(4):
        for v in cap.values():
            v.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        _everything(F, {**other_in, **other}, ows)    # eager work beside the replay
        torch.cuda.synchronize()
        for k in eager:
            assert torch.equal(cap[k], eager[k]), (rep, k)


def test_row_operators_on_another_stream_and_twice(F):
    """A side stream gives the same bits as the current one, twice."""
    ins, first = _tensors(F, 513, 770, 11)
    ws = dict(amax=F.workspace(), ln=F.layernorm_workspace(513, 770), moe=F.moe_workspace(1026, 8))
    _everything(F, {**ins, **first}, ws)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(2):
        _, again = _tensors(F, 513, 770, 11)
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            _everything(F, {**ins, **again}, ws)
        s.synchronize()
        for k in first:
            assert torch.equal(first[k], again[k]), k


def test_more_than_2_31_elements(F):
    """Offsets past 32 bits: the last rows of tensors of 2^31 + 2^21 elements
    equal a call on those rows alone."""
    rows, cols, n = (1 << 16) + 64, 32768, 8
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device=DEV)
    x[-n:] = torch.randn((n, cols), generator=g, device=DEV).bfloat16()
    x[:-n] = 1.5
    tail = x[-n:].contiguous()
    w = torch.ones(cols, dtype=torch.bfloat16, device=DEV)

    def run(v):
        r = v.shape[0]
        y, dx = (torch.empty_like(v) for _ in range(2))
        mean, rstd = (torch.empty(r, device=DEV) for _ in range(2))
        q = torch.empty((r, cols), dtype=torch.uint8, device=DEV)
        s = torch.empty((r, cols // 128), device=DEV)
        dg, db = (torch.empty(cols, device=DEV) for _ in range(2))
        F.fp8_layernorm_fwd(v, w, w, 1e-5, y, mean, rstd, xhat=F.cast_out(q, 0, BLOCK, s))
        F.fp8_layernorm_bwd(v, None, None, rstd, w, dx, dg, db, xhat=F.operand(q, 0, BLOCK, s))
        out = [t[-n:].clone() for t in (y, dx, q, s)]
        F.fp8_act_fwd(v, F.ACT_GELU, False, y, ckpt=F.cast_out(q, 0, BLOCK, s))
        F.fp8_act_bwd(v, F.operand(q, 0, BLOCK, s), F.ACT_GELU, False, dx)
        out += [t[-n:].clone() for t in (y, dx, q, s)]
        pos = torch.arange(r, dtype=torch.int32, device=DEV).view(r, 1)
        off = torch.tensor([0, r], dtype=torch.int32, device=DEV)
        F.fp8_moe_dispatch(v, pos, pos.view(-1), off, dx)
        F.fp8_moe_combine(dx, pos, None, y)
        out += [t[-n:].clone() for t in (dx, y)]
        return out
    for i, (a, b) in enumerate(zip(run(x), run(tail))):
        assert torch.equal(a, b), i
