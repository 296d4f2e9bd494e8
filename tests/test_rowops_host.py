"""The row operators on the host: their reference gradients against
differences, and what the C entry points and the binding refuse (before
anything is launched; the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

from tests import rowop_reference as R

NULL, SHAPE, ALIGN, UNSUP = 1, 2, 3, 4
P, PU = 0x10000, 0x10001


@pytest.fixture(scope="module")
def F():
    from scaled_fp8_gemm_amd import fp8sg
    fp8sg.lib()
    return fp8sg


# ------------------------------------------------ formulas and differences
# central differences in 64 bits with step s: error ~ s^2 (third derivative)
# + 2^-53 / s relative to the values, about 1e-9 here at s = 1e-5
STEP, DIFF = 1e-5, 1e-7


def _difference(f, x):
    g = torch.empty_like(x)
    flat = x.view(-1)
    for i in range(flat.numel()):
        v = flat[i].item()
        flat[i] = v + STEP
        up = f()
        flat[i] = v - STEP
        down = f()
        flat[i] = v
        g.view(-1)[i] = (up - down) / (2 * STEP)
    return g


def test_layernorm_gradient_against_differences():
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(3, 7, generator=g, dtype=torch.float64) for _ in range(2))
    gamma, beta = (torch.randn(7, generator=g, dtype=torch.float64) for _ in range(2))
    f = lambda: (R.ln_fwd(x, gamma, beta, 1e-5)[3] * dy).sum().item()  # noqa: E731
    _, rstd, xhat, _ = R.ln_fwd(x, gamma, beta, 1e-5)
    dx, dgamma, dbeta = R.ln_bwd(dy, xhat, rstd, gamma)
    for got, var in ((dx, x), (dgamma, gamma), (dbeta, beta)):
        assert torch.allclose(got, _difference(f, var), rtol=0, atol=DIFF * 10)


@pytest.mark.parametrize("act", [0, 1, 2])
def test_activation_gradient_against_differences(act):
    h = torch.linspace(-7, 7, 29, dtype=torch.float64)
    p, d = R.act_parts(act, h)
    up, down = h + STEP, h - STEP
    diff = (up * R.act_parts(act, up)[0] - down * R.act_parts(act, down)[0]) / (2 * STEP)
    assert torch.allclose(d, diff, rtol=0, atol=DIFF)


# ------------------------------------------------ refusals of the C calls
def _cast(F, scaling=1, fmt=0, data=P, sinv=P, scale=P, amax=None):
    return ctypes.byref(F.CastOut(data, fmt, scaling, sinv, scale, amax))


def _op(F, scaling=1, fmt=0, data=P, s=P):
    return ctypes.byref(F.Operand(data, fmt, scaling, s))


def test_layernorm_fwd_refusals(F):
    def f(x=P, xt=0, g=P, b=P, wt=0, rows=4, cols=16, eps=1e-5, y=P, mean=P, rstd=P, yq=None,
          xhat=None, ws=None):
        return F.lib().fp8_layernorm_fwd(x, xt, g, b, wt, rows, cols, eps, y, mean, rstd, yq, xhat,
                                         ws, None)
    for k in ("x", "g", "b", "y", "mean", "rstd"):
        assert f(**{k: None}) == NULL, k
        assert f(**{k: PU}) == ALIGN, k
    assert f(xt=2) == UNSUP and f(wt=-1) == UNSUP
    assert f(rows=-1) == SHAPE and f(cols=0) == SHAPE and f(cols=32769) == SHAPE
    assert f(eps=-1.0) == SHAPE and f(eps=float("nan")) == SHAPE and f(eps=float("inf")) == SHAPE
    assert f(yq=_cast(F, 2)) == UNSUP                    # 128x128
    assert f(yq=_cast(F, 7)) == UNSUP and f(yq=_cast(F, fmt=3)) == UNSUP
    assert f(xhat=_cast(F, 3)) == UNSUP and f(xhat=_cast(F, 0)) == UNSUP
    assert f(yq=_cast(F, data=None)) == NULL and f(yq=_cast(F, sinv=None)) == NULL
    assert f(yq=_cast(F, 0, scale=None)) == NULL
    assert f(yq=_cast(F, 0, amax=P)) == NULL             # amax without a workspace
    assert f(yq=_cast(F, 0, amax=P), ws=P + 64) == ALIGN
    assert f(yq=_cast(F, data=PU)) == ALIGN and f(yq=_cast(F, sinv=P + 2)) == ALIGN


def test_layernorm_bwd_refusals(F):
    def f(dy=P, x=P, xt=0, mean=P, rstd=P, xhat=None, g=P, wt=0, rows=4, cols=16, dx=P, dg=P, db=P,
          ws=P):
        return F.lib().fp8_layernorm_bwd(dy, x, xt, mean, rstd, xhat, g, wt, rows, cols, dx, dg,
                                         db, ws, None)
    for k in ("dy", "x", "mean", "rstd", "g", "dx", "dg", "db", "ws"):
        assert f(**{k: None}) == NULL, k
        assert f(**{k: PU}) == ALIGN, k
    assert f(xhat=_op(F)) == NULL                        # both x and xhat
    assert f(x=None, mean=None, xhat=_op(F, 3)) == UNSUP
    assert f(x=None, mean=None, xhat=_op(F, data=None)) == NULL
    assert f(x=None, mean=None, xhat=_op(F, s=P + 2)) == ALIGN
    assert f(xt=5) == UNSUP and f(rows=-1) == SHAPE and f(cols=0) == SHAPE
    assert f(cols=1 << 20) == SHAPE
    assert f(ws=P + 16) == ALIGN
    b = F.lib().fp8_layernorm_workspace_bytes
    assert b(0, 16) == 0 and b(4, 0) == 0 and b(-1, 16) == 0 and b(4, 1 << 20) == 0
    assert b(1, 100) >= 2 * 100 * 4


def test_activation_refusals(F):
    def f(h=P, act=0, gated=0, rows=4, cols=16, y=P, yq=None, ck=None, ws=None):
        return F.lib().fp8_act_fwd(h, act, gated, rows, cols, y, yq, ck, ws, None)
    assert f(h=None) == NULL and f(y=None) == NULL
    assert f(act=3) == UNSUP and f(act=-1) == UNSUP and f(gated=2) == UNSUP
    assert f(rows=-1) == SHAPE and f(cols=-1) == SHAPE
    assert f(h=PU) == ALIGN and f(y=PU) == ALIGN
    assert f(yq=_cast(F, 2)) == UNSUP and f(ck=_cast(F, 3)) == UNSUP
    assert f(yq=_cast(F, 0, amax=P)) == NULL

    def b(dy=P, h=P, ck=None, act=0, gated=0, rows=4, cols=16, dh=P, y=None):
        return F.lib().fp8_act_bwd(dy, h, ck, act, gated, rows, cols, dh, y, None)
    for k in ("dy", "h", "dh"):
        assert b(**{k: None}) == NULL, k
        assert b(**{k: PU}) == ALIGN, k
    assert b(y=PU) == ALIGN and b(ck=_op(F)) == NULL and b(h=None, ck=_op(F, 0)) == UNSUP
    assert b(act=9) == UNSUP and b(rows=-2) == SHAPE


def test_checkpoint_refusals(F):
    s, ld = F.lib().fp8_checkpoint_save, F.lib().fp8_checkpoint_load
    assert s(P, 4, 16, None, None) == NULL and s(None, 4, 16, _cast(F), None) == NULL
    assert s(P, 4, 16, _cast(F, 3), None) == UNSUP and s(P, -4, 16, _cast(F), None) == SHAPE
    assert s(PU, 4, 16, _cast(F), None) == ALIGN
    assert ld(None, 4, 16, P, None) == NULL and ld(_op(F), 4, 16, None, None) == NULL
    assert ld(_op(F, 2), 4, 16, P, None) == UNSUP and ld(_op(F), 4, -1, P, None) == SHAPE
    assert ld(_op(F), 4, 16, PU, None) == ALIGN


def test_moe_refusals(F):
    L = F.lib()

    def s(e=P, tokens=4, k=2, experts=8, pad=16, rows=128, off=P, cnt=P, pos=P, src=P, ws=P):
        return L.fp8_moe_sort(e, tokens, k, experts, pad, rows, off, cnt, pos, src, ws, None)
    for n in ("e", "off", "cnt", "pos", "src", "ws"):
        assert s(**{n: None}) == NULL, n
        assert s(**{n: PU}) == ALIGN, n
    assert L.fp8_moe_rows(8, 8, 16) == 128
    assert s(rows=127) == SHAPE and s(k=0) == SHAPE and s(experts=0) == SHAPE
    assert s(experts=1025) == SHAPE and s(pad=0) == SHAPE and s(tokens=-1) == SHAPE
    assert s(rows=1 << 31) == SHAPE and s(tokens=1 << 30, k=2) == SHAPE
    assert s(pad=(1 << 31) - 1) == SHAPE          # the padded rows pass 2^31
    assert L.fp8_moe_rows(10, 4, 1) == 10 and L.fp8_moe_rows(0, 4, 128) == 0
    assert L.fp8_moe_rows(3, 100, 128) == 3 * 128 and L.fp8_moe_rows(1000, 4, 128) == 1408
    assert L.fp8_moe_rows(-1, 4, 1) == 0 and L.fp8_moe_workspace_bytes(10, 0) == 0

    def d(x=P, tokens=4, k=2, cols=16, pos=P, src=P, off=P, experts=8, rows=128, xs=P, xq=None):
        return L.fp8_moe_dispatch(x, tokens, k, cols, pos, src, off, experts, rows, xs, xq, None)
    for n in ("x", "pos", "src", "off", "xs"):
        assert d(**{n: None}) == NULL, n
        assert d(**{n: PU}) == ALIGN, n
    assert d(cols=-1) == SHAPE and d(k=0) == SHAPE and d(experts=0) == SHAPE and d(rows=-1) == SHAPE
    assert d(xq=_cast(F, 2)) == UNSUP and d(xq=_cast(F, 0, amax=P)) == UNSUP

    def c(ys=P, pos=P, w=P, tokens=4, k=2, cols=16, rows=128, y=P):
        return L.fp8_moe_combine(ys, pos, w, tokens, k, cols, rows, y, None)
    for n in ("ys", "pos", "y"):
        assert c(**{n: None}) == NULL, n
        assert c(**{n: PU}) == ALIGN, n
    assert c(w=PU) == ALIGN and c(k=0) == SHAPE and c(rows=1 << 31) == SHAPE

    def b(dy=P, ys=P, w=P, pos=P, src=P, off=P, tokens=4, k=2, cols=16, experts=8, rows=128, dys=P,
          dw=P):
        return L.fp8_moe_combine_bwd(dy, ys, w, pos, src, off, tokens, k, cols, experts, rows, dys,
                                     dw, None)
    for n in ("dy", "ys", "w", "pos", "src", "off", "dys", "dw"):
        assert b(**{n: None}) == NULL, n
        assert b(**{n: PU}) == ALIGN, n
    assert b(tokens=-1) == SHAPE and b(experts=2000) == SHAPE


def test_binding_refuses_host_and_wrong_tensors(F):
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    f = torch.zeros(16)
    with pytest.raises(ValueError, match="on the GPU"):
        F.fp8_layernorm_fwd(x, f, f, 1e-5, x, f, f)
    with pytest.raises(ValueError, match="beta has dtype"):
        F.fp8_layernorm_fwd(x, f, f.bfloat16(), 1e-5, x, f, f)
    with pytest.raises(ValueError, match="must be even"):
        F.fp8_act_fwd(torch.zeros(4, 15, dtype=torch.bfloat16), 2, True, x)
    with pytest.raises(ValueError, match="2-D"):
        F.fp8_moe_combine(x, torch.zeros(4, dtype=torch.int32), None, x)


def test_cast_out_keeps_its_tensors(F):
    import gc
    import weakref
    t = [torch.zeros(64, dtype=torch.uint8), torch.ones(1), torch.ones(1), torch.ones(1)]
    refs = [weakref.ref(v) for v in t]
    o = F.cast_out(t[0], F.E4M3, F.SCALE_TENSOR, t[1], t[2], t[3])
    del t
    gc.collect()
    assert all(r() is not None for r in refs)
    assert o.amax == refs[3]().data_ptr()
