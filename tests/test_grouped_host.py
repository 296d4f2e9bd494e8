"""What the products by expert and with 4-bit operands refuse, on the host
before anything is launched (the pointers are never dereferenced)."""
import ctypes

import pytest
import torch

NULL, SHAPE, ALIGN, UNSUP = 1, 2, 3, 4
P, PU = 0x10000, 0x10001
TENSOR, BLOCK, SQUARE, MX = 0, 1, 2, 3
E2M1 = 4


@pytest.fixture(scope="module")
def F():
    from scaled_fp8_gemm_amd import fp8sg
    fp8sg.lib()
    return fp8sg


def op(F, fmt=0, scaling=TENSOR, data=P, s=P):
    return ctypes.byref(F.Operand(data, fmt, scaling, s))


@pytest.mark.parametrize("name", ["fprop", "dgrad", "wgrad", "wgrad_f32"])
def test_grouped(F, name):
    fn = getattr(F.lib(), "fp8_gemm_grouped_" + name)
    tail = (0, None) if name == "wgrad_f32" else (None,)
    depth = name.startswith("wgrad")

    def f(a=None, b=None, off=P, experts=8, rows=256, N=256, K=256, c=P):
        return fn(a or op(F), b or op(F), off, experts, rows, N, K, c, *tail)
    assert fn(None, op(F), P, 8, 256, 256, 256, P, *tail) == NULL
    assert fn(op(F), None, P, 8, 256, 256, 256, P, *tail) == NULL
    assert f(off=None) == NULL and f(c=None) == NULL
    for k in ("data", "s"):
        assert f(a=op(F, **{k: None})) == NULL and f(b=op(F, **{k: None})) == NULL
        assert f(a=op(F, **{k: PU})) == ALIGN and f(b=op(F, **{k: PU})) == ALIGN
    assert f(off=P + 2) == ALIGN and f(c=PU) == ALIGN
    for experts in (0, -1, 1025):
        assert f(experts=experts) == SHAPE
    assert f(rows=-1) == SHAPE and f(N=-1) == SHAPE and f(K=-16) == SHAPE
    assert f(rows=1 << 31) == SHAPE and f(N=1 << 31) == SHAPE
    assert f(a=op(F, 7)) == UNSUP and f(b=op(F, 2)) == UNSUP and f(a=op(F, 0, 9)) == UNSUP
    # families do not mix
    assert f(a=op(F, 0, BLOCK)) == UNSUP and f(a=op(F, 0, MX), b=op(F, 0, BLOCK)) == UNSUP
    assert f(a=op(F, 0, SQUARE), b=op(F, 0, BLOCK)) == UNSUP      # rows in 128x128 blocks
    # 4 bits: the second or both, MX, and not the weight gradients
    assert f(a=op(F, E2M1, MX), b=op(F, 0, MX)) == UNSUP
    assert f(b=op(F, E2M1)) == UNSUP and f(a=op(F, 0, BLOCK), b=op(F, E2M1, BLOCK)) == UNSUP
    if depth:
        assert f(a=op(F, E2M1, MX), b=op(F, E2M1, MX)) == UNSUP
        assert f(a=op(F, 0, BLOCK), b=op(F, 0, SQUARE)) == UNSUP
        assert f(rows=24) == ALIGN
        assert f(a=op(F, 0, MX), b=op(F, 0, MX), rows=160) == SHAPE
        assert f(a=op(F, 0, BLOCK), b=op(F, 0, BLOCK), rows=160) == SHAPE
        assert f(rows=(1 << 23) + 16) == SHAPE
        assert f(experts=1024, N=1 << 20, K=1 << 20) == SHAPE     # too many tiles
        assert f(a=op(F, 0, MX, s=P + 2), b=op(F, 0, MX)) == ALIGN
    else:
        con, n = ("N", "K") if name == "dgrad" else ("K", "N")
        assert f(**{con: 24}) == ALIGN and f(**{con: (1 << 23) + 16}) == SHAPE
        assert f(a=op(F, 0, MX), b=op(F, 0, MX), **{con: 48}) == SHAPE
        assert f(a=op(F, 0, BLOCK), b=op(F, 0, BLOCK), **{con: 64}) == SHAPE
        assert f(a=op(F, 0, BLOCK), b=op(F, 0, SQUARE), **{n: 200}) == SHAPE
        assert f(rows=1 << 30, **{n: 1 << 30}) == SHAPE           # too many tiles
    if name == "wgrad_f32":
        assert fn(op(F), op(F), P, 8, 256, 256, 256, P, 2, None) == UNSUP


def test_fp4_operands(F):
    g = F.lib().fp8_gemm_fprop
    x4, x8, w4 = op(F, E2M1, MX), op(F, 0, MX), op(F, E2M1, MX)
    assert g(x4, x8, 16, 16, 64, P, None) == UNSUP               # the first alone
    assert g(op(F, E2M1), op(F, E2M1), 16, 16, 64, P, None) == UNSUP
    assert g(op(F, 0, TENSOR), w4, 16, 16, 64, P, None) == UNSUP
    assert g(op(F, 0, BLOCK), op(F, E2M1, BLOCK), 16, 16, 128, P, None) == UNSUP
    assert g(x8, w4, 16, 16, 48, P, None) == SHAPE and g(x4, w4, -1, 16, 64, P, None) == SHAPE
    assert g(x8, w4, 16, 16, 64, PU, None) == ALIGN
    assert g(x8, op(F, E2M1, MX, data=PU), 16, 16, 64, P, None) == ALIGN
    assert g(x8, op(F, E2M1, MX, data=None), 16, 16, 64, P, None) == NULL
    ff = F.lib().fp8_gemm_fprop_fused
    assert ff(x8, w4, 16, 16, 64, P, E2M1, P, P, None, None, None) == UNSUP      # y in 4 bits
    # formats of 8 bits elsewhere
    assert F.lib().fp8_quantize_mx(P, 4, 64, E2M1, P, P, None) == UNSUP
    assert F.lib().fp8_quantize_tensor(P, 4, 64, E2M1, P, P, None, None, None, None) == UNSUP
    assert F.lib().fp8_convert_f32(P, 4, E2M1, P, None) == UNSUP


def test_binding(F):
    u = torch.zeros(64, 32, dtype=torch.uint8)
    o = F.operand(u, 0, MX, u)
    off, y = torch.zeros(3, dtype=torch.int32), torch.zeros(64, 32, dtype=torch.bfloat16)
    for fn in (F.fp8_gemm_grouped_fprop, F.fp8_gemm_grouped_dgrad, F.fp8_gemm_grouped_wgrad,
               F.fp8_gemm_grouped_wgrad_f32):
        with pytest.raises(ValueError, match="on the GPU"):
            fn(o, o, off, 2, 64, 32, 32, y)
        with pytest.raises(TypeError, match="must be an operand"):
            fn(u, o, off, 2, 64, 32, 32, y)


@pytest.mark.gpu
def test_binding_checks_sizes(F):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    x = F.operand(u8(64, 64), 0, MX, u8(64, 2))
    w4 = F.operand(u8(96, 32), E2M1, MX, u8(96, 2))
    off, y = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(64, 48, device="cuda")
    y = y.bfloat16()
    F.fp8_gemm_grouped_fprop(x, w4, off, 2, 64, 48, 64, y)
    f = F.fp8_gemm_grouped_fprop
    for name, args in (("offsets", (x, w4, off[:2], 2, 64, 48, 64, y)),
                       ("w.data", (x, w4, off, 2, 64, 49, 64, y)),
                       ("x.data", (x, w4, off, 2, 65, 48, 64, y)),
                       ("y holds", (x, w4, off, 2, 64, 48, 64, y[:60].contiguous()))):
        with pytest.raises(ValueError, match=name):
            f(*args)
    xt = F.operand(u8(64, 64), 0, TENSOR, torch.ones(1, device="cuda"))
    wt = F.operand(u8(96, 64), 0, TENSOR, torch.ones(1, device="cuda"))
    with pytest.raises(ValueError, match="w.scale_inv"):       # one for each expert
        f(xt, wt, off, 2, 64, 48, 64, y)
