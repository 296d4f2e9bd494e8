"""Quantised operands as FP64 values, and products checked against them under
the error model of gpu_helpers (the MFMA's truncation within a step of 128 K,
FP32 sums, one BF16 rounding)."""
import numpy as np
import torch

from tests.gpu_helpers import bits16, compare, truncation_per_step
from tests.rms_reference import mx4, mx4_values, pack

FP8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}
TENSOR, BLOCK, SQUARE, MX = 0, 1, 2, 3
E2M1 = 4


def scales(g, scaling, rows, k, tensors=1):
    """Random scales of an operand [rows][k]."""
    def spread(*shape):
        return torch.exp2(torch.randint(-3, 4, shape, generator=g).float()) * (
            1 + torch.rand(shape, generator=g))
    if scaling == TENSOR:
        return spread(tensors)
    if scaling == BLOCK:
        return spread(rows, k // 128)
    if scaling == SQUARE:
        return spread(rows // 128, k // 128)
    return torch.randint(121, 133, (rows, k // 32), generator=g).to(torch.uint8)


def operand(seed, rows, k, fmt, scaling, tensors=1):
    """(bytes, scales) of a random operand: normal values rounded to fmt."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randn(rows, k, generator=g)
    if fmt == E2M1:
        q = torch.zeros(rows, k // 2, dtype=torch.uint8)
        if rows * k:             # every code among them
            q = pack(mx4((v * 2).clamp(-6, 6).bfloat16())[0])
    else:
        q = v.to(FP8[fmt]).view(torch.uint8)
    return q, scales(g, scaling, rows, k, tensors)


def values(q, s, fmt, scaling, rows_per_tensor=None):
    """What the operand stands for, FP64; rows_per_tensor: rows of each scale
    under per-tensor scaling of several tensors."""
    q, s = q.cpu(), s.cpu()
    if fmt == E2M1:
        return mx4_values(q, s)
    v = q.view(FP8[fmt]).double()
    if scaling == TENSOR:
        f = s.double()
        return v * (f.repeat_interleave(rows_per_tensor)[:, None] if rows_per_tensor else f)
    if scaling == MX:
        f = torch.where(s == 255, float("nan"), torch.exp2(s.double() - 127))
        return v * f.repeat_interleave(32, 1)
    f = s.double().repeat_interleave(128, 1)
    return v * (f.repeat_interleave(128, 0) if scaling == SQUARE else f)


def parts(a, b):
    """Exact a b^T, the sum of its terms' magnitudes and the truncation bound.
    Scales are folded into the values; one that is no power of two may move a
    step's largest product past a power of two, hence the factor 2."""
    an, bn = torch.nan_to_num(a, nan=0.0), torch.nan_to_num(b, nan=0.0)
    t = truncation_per_step(an.numpy(), bn.numpy())
    return a @ b.t(), an.abs() @ bn.abs().t(), 2 * t.sum(-1)


def check(orc, y, a, b, label):
    """BF16 y against a b^T."""
    if y.numel() == 0:
        return
    want, mag, t = parts(a, b)
    steps = -(-a.shape[1] // 128)
    compare(orc, bits16(y), want.numpy(), mag.numpy(), t, steps, label)


def check_f32(y, old, a, b, label):
    """FP32 y against old + a b^T."""
    want, mag, t = parts(a, b)
    want = want + old.cpu().double()
    got = y.cpu().double()
    steps = -(-a.shape[1] // 128)
    bound = (torch.from_numpy(np.asarray(t)) + (3 * steps + 4) * 2.0 ** -24 * mag
             + 2.0 ** -24 * (got.abs() + old.cpu().double().abs()) + 2.0 ** -120)
    bad = (got - want).abs() > bound
    assert not bad.any(), (label, int(bad.sum()), bad.nonzero()[0])
