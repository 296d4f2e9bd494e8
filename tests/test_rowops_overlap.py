"""Row operators whose output takes the place of an input: the same bits as
into another tensor where that is allowed, at widths that end in a slot of
another group of lanes, and refused elsewhere."""
import ctypes

import pytest
import torch

from scaled_fp8_gemm_amd import fp8sg as F

UNSUP = 4
P = 0x10000


def test_refused():
    """Addresses of no memory, each another but for the pair that clashes."""
    L, at = F.lib(), iter(range(0x100000, 1 << 30, 0x1000))
    n = lambda: next(at)  # noqa: E731
    out = lambda q: ctypes.byref(F.CastOut(q, 0, 1, n(), None, None))  # noqa: E731
    held = lambda q: ctypes.byref(F.Operand(q, 0, 1, n()))  # noqa: E731
    a = [n() for _ in range(40)]
    lnf = lambda x, xt, y, yq=None, xh=None: L.fp8_layernorm_fwd(  # noqa: E731
        x, xt, a[1], a[2], 0, 4, 16, 1e-5, y, a[3], a[4], yq, xh, None, None)
    assert lnf(P, 1, P) == UNSUP
    assert lnf(P, 0, a[5], yq=out(P)) == UNSUP and lnf(P, 0, a[5], xh=out(P)) == UNSUP
    assert L.fp8_layernorm_bwd(P, a[5], 1, a[1], a[2], None, a[3], 0, 4, 16, P, a[6], a[7],
                               a[8], None) == UNSUP
    assert L.fp8_layernorm_bwd(a[5], None, 0, None, a[2], held(P), a[3], 0, 4, 16, P, a[6], a[7],
                               a[8], None) == UNSUP
    actf = lambda gated, y, yq=None, ck=None: L.fp8_act_fwd(P, 2, gated, 4, 16, y, yq, ck,  # noqa: E731
                                                            None, None)
    assert actf(1, P) == UNSUP
    assert actf(0, a[5], yq=out(P)) == UNSUP and actf(1, a[5], ck=out(P)) == UNSUP
    actb = lambda dy, h, ck, gated, dh, y: L.fp8_act_bwd(dy, h, ck, 2, gated, 4, 16, dh, y,  # noqa: E731
                                                         None)
    assert actb(P, a[1], None, 1, P, None) == UNSUP      # gated: dh is wider than dy
    assert actb(a[1], P, None, 1, a[2], P) == UNSUP      # and y narrower than h
    assert actb(a[1], None, held(P), 0, P, None) == UNSUP
    assert actb(a[1], None, held(P), 0, a[2], P) == UNSUP
    assert L.fp8_checkpoint_save(P, 4, 16, out(P), None) == UNSUP
    assert L.fp8_checkpoint_load(held(P), 4, 16, P, None) == UNSUP
    disp = lambda xs, xq: L.fp8_moe_dispatch(P, 4, 2, 16, a[1], a[2], a[3], 8, 128, xs, xq,  # noqa: E731
                                             None)
    assert disp(P, None) == UNSUP and disp(a[5], out(P)) == UNSUP
    assert L.fp8_moe_combine(P, a[1], a[2], 4, 2, 16, 128, P, None) == UNSUP
    comb = lambda dy, ys: L.fp8_moe_combine_bwd(dy, ys, a[1], a[2], a[3], a[4], 4, 2, 16, 8,  # noqa: E731
                                                128, P, a[5], None)
    assert comb(P, a[6]) == UNSUP and comb(a[6], P) == UNSUP


# one to seven columns in a tile of their own, in a slot of a tile, none
WIDTHS = [1, 7, 9, 129, 133, 250, 513, 1001, 1025, 1030, 4096, 4101, 12289]


@pytest.mark.gpu
@pytest.mark.parametrize("cols", WIDTHS)
def test_in_place(cols):
    rows = 900
    g = torch.Generator(device="cuda").manual_seed(cols)
    new = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()  # noqa: E731
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    x, dy, w = new(rows, cols), new(rows, cols), torch.ones(cols, device="cuda")
    m, r = f(rows), f(rows)

    def same(call, *outs_and_ins):
        """call(*tensors): the outputs' own tensors, then inputs in their place."""
        own = [torch.empty_like(t) for t in outs_and_ins]
        call(*own)
        for i, t in enumerate(outs_and_ins):
            want = own[i].clone()
            others = [torch.empty_like(v) for v in outs_and_ins]
            others[i] = t
            keep = t.clone()
            call(*others)
            assert torch.equal(t.view(torch.int16), want.view(torch.int16)), i
            t.copy_(keep)
    same(lambda y: F.fp8_layernorm_fwd(x, w, w, 1e-5, y, m, r), x)
    F.fp8_layernorm_fwd(x, w, w, 1e-5, torch.empty_like(x), m, r)
    for t in (x, dy):
        same(lambda dx: F.fp8_layernorm_bwd(dy, x, m, r, w, dx, f(cols), f(cols)), t)
    x32 = x.float()
    d1, d2 = torch.empty_like(x32), x32.clone()
    F.fp8_layernorm_bwd(dy, x32, m, r, w, d1, f(cols), f(cols))
    F.fp8_layernorm_bwd(dy, d2, m, r, w, d2, f(cols), f(cols))
    assert torch.equal(d1, d2)
    for act in (F.ACT_GELU, F.ACT_GELU_TANH, F.ACT_SILU):
        same(lambda y: F.fp8_act_fwd(x, act, False, y), x)
        for t, u in ((x, dy), (dy, x)):
            same(lambda dh, y: F.fp8_act_bwd(dy, x, act, False, dh, y=y), t, u)
        h = new(rows, 2 * cols)
        same(lambda dh, y: F.fp8_act_bwd(dy, h, act, True, dh, y=y), h, dy)
