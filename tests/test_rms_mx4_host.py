"""RMS norm and the 4-bit cast on the host: reference gradients against
differences, the 4-bit rule against a search, and refusals (before anything
is launched; the pointers are never dereferenced)."""
import ctypes
import itertools

import pytest
import torch

from tests import rms_reference as M
from tests.test_rowops_host import DIFF, _difference

NULL, SHAPE, ALIGN, UNSUP = 1, 2, 3, 4
P, PU = 0x10000, 0x10001


@pytest.fixture(scope="module")
def F():
    from scaled_fp8_gemm_amd import fp8sg
    fp8sg.lib()
    return fp8sg


def test_gradient_against_differences():
    g = torch.Generator().manual_seed(3)
    h, dy, dres = (torch.randn(3, 7, generator=g, dtype=torch.float64) for _ in range(3))
    gamma = torch.randn(7, generator=g, dtype=torch.float64)
    f = lambda: ((M.rms_fwd(h, gamma, 1e-5)[2] * dy).sum() + (h * dres).sum()).item()  # noqa: E731
    rstd, xhat, _ = M.rms_fwd(h, gamma, 1e-5)
    dx, dgamma = M.rms_bwd(dy, xhat, rstd, gamma, dres)
    for got, var in ((dx, h), (dgamma, gamma)):
        assert torch.allclose(got, _difference(f, var), rtol=0, atol=DIFF * 10)


def test_mx4_rule_against_a_search():
    """The least exponent whose grid reaches the largest value, the nearest
    grid value, and of two as near the one with the even code."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(40, 32, generator=g).bfloat16()
    x[:8] = (torch.randint(-24, 25, (8, 32), generator=g) / 4).bfloat16()
    code, byte = M.mx4(x)
    for r in range(40):
        v = x[r].double()
        e = next(e for e in itertools.count(-140) if v.abs().max() <= 6 * 2.0 ** e)
        assert byte[r, 0] == e + 127
        for i in range(32):
            d = [abs(abs(v[i].item()) - t * 2.0 ** e) for t in M.E2M1]
            near = [k for k in range(8) if d[k] == min(d)]
            want = min(near, key=lambda k: k % 2)
            assert code[r, i] % 8 == want
    q = M.pack(code)
    assert torch.equal(M.unpack(q), code)


def _cast(F, scaling=1, fmt=0, data=0x30000, sinv=P, scale=P, amax=None):
    return ctypes.byref(F.CastOut(data, fmt, scaling, sinv, scale, amax))


def _op(F, scaling=1, fmt=0, data=0x30000, s=P):
    return ctypes.byref(F.Operand(data, fmt, scaling, s))


def test_forward_refusals(F):
    def f(x=P, xt=0, d=0x20000, g=P, wt=0, rows=4, cols=16, eps=1e-5, h=0x40000, y=0x50000, rstd=P,
          yq=None, xhat=None, ws=None):
        return F.lib().fp8_rmsnorm_fwd(x, xt, d, g, wt, rows, cols, eps, h, y, rstd, yq, xhat, ws,
                                       None)
    for k in ("x", "g", "rstd"):
        assert f(**{k: None}) == NULL, k
    assert f(h=None, y=None) == NULL                     # no output
    for k in ("x", "d", "g", "h", "y", "rstd"):
        assert f(**{k: PU}) == ALIGN, k
    assert f(xt=2) == UNSUP and f(wt=-1) == UNSUP
    assert f(rows=-1) == SHAPE and f(cols=0) == SHAPE and f(cols=32769) == SHAPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert f(eps=eps) == SHAPE
    assert f(yq=_cast(F, 2)) == UNSUP and f(yq=_cast(F, fmt=3)) == UNSUP
    assert f(yq=_cast(F, 3, fmt=4)) == UNSUP             # E2M1
    assert f(xhat=_cast(F, 3)) == UNSUP and f(xhat=_cast(F, 0)) == UNSUP
    assert f(yq=_cast(F, data=None)) == NULL and f(yq=_cast(F, sinv=None)) == NULL
    assert f(yq=_cast(F, 0, scale=None)) == NULL and f(yq=_cast(F, 0, amax=P)) == NULL
    assert f(yq=_cast(F, 0, amax=P), ws=P + 64) == ALIGN
    # outputs over inputs of another shape or type, or over each other
    assert f(xt=1, h=0x20000) == UNSUP and f(xt=1, y=P) == UNSUP and f(y=0x40000) == UNSUP
    for at in (P, 0x20000):
        assert f(yq=_cast(F, data=at)) == UNSUP and f(xhat=_cast(F, data=at)) == UNSUP


def test_backward_refusals(F):
    def f(dy=P, h=0x20000, xt=0, rstd=P, xhat=None, g=P, wt=0, res=0x50000, rows=4, cols=16,
          dx=0x40000, dg=P, ws=P):
        return F.lib().fp8_rmsnorm_bwd(dy, h, xt, rstd, xhat, g, wt, res, rows, cols, dx, dg, ws,
                                       None)
    for k in ("dy", "h", "rstd", "g", "dx", "dg", "ws"):
        assert f(**{k: None}) == NULL, k
    for k in ("dy", "h", "rstd", "g", "res", "dx", "dg", "ws"):
        assert f(**{k: PU}) == ALIGN, k
    assert f(xhat=_op(F)) == NULL                        # both h and xhat
    assert f(h=None, xhat=_op(F, 3)) == UNSUP and f(h=None, xhat=_op(F, fmt=4)) == UNSUP
    assert f(h=None, xhat=_op(F, data=None)) == NULL
    assert f(h=None, xhat=_op(F, s=P + 2)) == ALIGN
    assert f(xt=5) == UNSUP and f(rows=-1) == SHAPE and f(cols=0) == SHAPE
    assert f(cols=1 << 20) == SHAPE and f(ws=P + 16) == ALIGN
    assert f(xt=1, dx=P) == UNSUP and f(h=None, xhat=_op(F), dx=0x30000) == UNSUP
    b = F.lib().fp8_rmsnorm_workspace_bytes
    assert b(0, 16) == 0 and b(4, 0) == 0 and b(-1, 16) == 0 and b(4, 1 << 20) == 0
    assert b(1, 100) >= 400 and b(10 ** 6, 100) == 256 * 400


def test_mx4_refusals(F):
    q, t, d = (getattr(F.lib(), "fp8_" + n) for n in ("quantize_mx4", "quantize_mx4_t",
                                                      "dequantize_mx4"))
    assert q(P, 4, 48, P, P, None) == SHAPE and q(P, -4, 32, P, P, None) == SHAPE
    for k in range(3):
        a = [P, P, P]
        a[k] = None
        assert q(a[0], 4, 64, a[1], a[2], None) == NULL
        assert d(a[0], a[1], 4, 64, a[2], None) == NULL
    assert q(PU, 4, 64, P, P, None) == ALIGN and q(P, 4, 64, PU, P, None) == ALIGN
    assert d(PU, P, 4, 64, P, None) == ALIGN and d(P, P, 4, 64, PU, None) == ALIGN
    assert d(P, P, 4, 48, P, None) == SHAPE and d(P, P, 4, -32, P, None) == SHAPE
    assert t(P, 48, 64, P, P, P, P, None) == SHAPE and t(P, 64, 48, P, P, P, P, None) == SHAPE
    assert t(P, 64, 64, None, P, P, P, None) == NULL and t(P, 64, 64, P, None, P, P, None) == NULL
    assert t(P, 64, 64, None, None, None, P, None) == NULL
    assert t(P, 64, 64, None, None, P, None, None) == NULL and t(None, 64, 64, P, P, P, P, None) == NULL
    for k in (PU,):
        assert t(k, 64, 64, P, P, P, P, None) == ALIGN and t(P, 64, 64, k, P, P, P, None) == ALIGN
        assert t(P, 64, 64, P, P, k, P, None) == ALIGN


def test_binding_refusals(F):
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    f, u = torch.zeros(32), torch.zeros(4, 16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="h has dtype"):
        F.fp8_rmsnorm_fwd(x, None, f, 1e-5, f, x, f)
    with pytest.raises(ValueError, match="dx has dtype"):
        F.fp8_rmsnorm_bwd(x, x, f, f, f.view(1, 32), x, f, workspace=u)
    with pytest.raises(TypeError, match="xhat must be an operand"):
        F.fp8_rmsnorm_bwd(x, None, f, f, None, x, f, xhat=u, workspace=u)
    with pytest.raises(ValueError, match="on the GPU"):
        F.fp8_rmsnorm_fwd(x, x, f, 1e-5, x, x, f)
    with pytest.raises(ValueError, match="on the GPU"):
        F.fp8_quantize_mx4(x, u, u)
    with pytest.raises(ValueError, match="2-D"):
        F.fp8_quantize_mx4_t(f, u, u, u, u)
    with pytest.raises(ValueError, match="on the GPU"):
        F.fp8_dequantize_mx4(u, u, 4, 32, x)
