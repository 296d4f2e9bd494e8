"""The row operators' formulas in 64 bits, elementary torch operations only,
and the error bounds their FP32 kernels are held to.

U = 2^-24 is FP32's half step.  A bound counts the kernel's roundings: a sum
of c values in chunks of at most 32 per thread, then a tree, is off by at
most 64 U sum |v|; v_exp, v_rcp and division are within 2 U of the value.
Rounding to the output's type adds half a step of it: 2^-8 of the value for
BF16, 2^-4 / 2^-3 for E4M3 / E5M2, and half the smallest step below its normal
range.
"""
import math

import torch

U = 2.0 ** -24
FMAX = {0: 448.0, 1: 57344.0}
HALF = {0: 2.0 ** -4, 1: 2.0 ** -3}          # of the value
TINY = {0: 2.0 ** -10, 1: 2.0 ** -17}        # half the smallest step
BF16 = 2.0 ** -8
FP8 = {0: torch.float8_e4m3fn, 1: torch.float8_e5m2}


# ------------------------------------------------------------ layer norm
def ln_fwd(x, gamma, beta, eps):
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / torch.sqrt((d * d).mean(1) + eps)
    xhat = d * rstd[:, None]
    return mean, rstd, xhat, xhat * gamma + beta


def ln_fwd_bounds(x, gamma, beta, mean, rstd, xhat):
    """Absolute bounds of mean, rstd, xhat, y."""
    mag = x.abs().mean(1)
    t_mean = 70 * U * mag
    # the deviations are off by t_mean + U |d| each; the variance by twice
    # that times its root, its own sum's 64 U and its square
    rel = 40 * U + rstd * t_mean + (rstd * t_mean) ** 2
    t_rstd = rstd * rel
    t_xhat = xhat.abs() * (rel + 4 * U)[:, None] + (rstd * t_mean * 1.01)[:, None]
    t_y = gamma.abs() * t_xhat + 3 * U * ((xhat * gamma).abs() + beta.abs())
    return t_mean, t_rstd, t_xhat, t_y


def ln_bwd(dy, xhat, rstd, gamma):
    g = dy * gamma
    c1, c2 = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
    dx = rstd[:, None] * (g - c1 - xhat * c2)
    return dx, (dy * xhat).sum(0), dy.sum(0)


def ln_bwd_bounds(dy, xhat, t_xhat, rstd, gamma):
    """t_xhat: how far the kernel's xhat may be off."""
    g = (dy * gamma).abs()
    xa = xhat.abs() + t_xhat
    t_c1 = 70 * U * g.mean(1, keepdim=True)
    t_c2 = 72 * U * (g * xa).mean(1, keepdim=True) + (g * t_xhat).mean(1, keepdim=True)
    c2 = (dy * gamma * xhat).mean(1, keepdim=True).abs()
    t_dx = rstd[:, None] * (6 * U * (g + g.mean(1, keepdim=True) + xa * c2) + t_c1 + xa * t_c2
                            + t_xhat * c2)
    rows = dy.shape[0]
    # rows are added one after the other within a workgroup (at most all of
    # them), then across workgroups
    t_dg = (rows + 80) * U * (dy.abs() * xa).sum(0) + (dy.abs() * t_xhat).sum(0)
    t_db = (rows + 80) * U * dy.abs().sum(0)
    return t_dx, t_dg, t_db


# ------------------------------------------------------------ activations
def act_parts(act, h):
    """(p, act') with act(h) = h p; act: 0 gelu, 1 gelu tanh, 2 silu."""
    if act == 2:
        p = torch.sigmoid(h)
        return p, p * (1 + h * (1 - p))
    if act == 0:
        p = 0.5 * torch.special.erfc(-h / math.sqrt(2))
        return p, p + h * torch.exp(-h * h / 2) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    p = torch.sigmoid(2 * a * (h + 0.044715 * h ** 3))
    return p, p + 2 * a * h * (1 + 3 * 0.044715 * h * h) * p * (1 - p)


def act_bounds(act, h):
    """Relative bound of p, absolute bound of act'."""
    p, d = act_parts(act, h)
    a = h.abs()
    if act == 2:
        rel, slope = (2 * a + 8) * U, torch.ones_like(h)
    elif act == 0:
        rel, slope = (2 * h * h + 40) * U, torch.zeros_like(h)
    else:
        k = math.sqrt(2 / math.pi)
        rel = (8 * k * (a + 0.044715 * a ** 3) + 10) * U
        slope = 2 * k * (1 + 3 * 0.044715 * h * h)
    return rel, 8 * (rel + 4 * U) * (p + (d - p).abs() + a * slope * p)


# ------------------------------------------------------------ casts
def tiles(v, b):
    r, c = v.shape
    n = -(-c // b)
    return torch.nn.functional.pad(v, (0, n * b - c)).view(r, n, b)


def held_values(q, scale_inv, fmt):
    """Bytes and 1x128 scales -> the values they stand for."""
    r, c = q.shape
    v = tiles(q.cpu().view(FP8[fmt]).double(), 128) * scale_inv.cpu().double().view(r, -1, 1)
    return v.view(r, -1)[:, :c]


def check_close(got, want, tol, label):
    got = got.detach().cpu().double().reshape(want.shape)
    bad = ~((got - want).abs() <= tol)
    bad &= ~(torch.isnan(got) & torch.isnan(want))
    bad &= ~(torch.isinf(want) & (got == want))
    n = int(bad.sum())
    if n:
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError(f"{label}: {n} of {bad.numel()} off; first at {i}: got "
                             f"{got.reshape(-1)[i].item()!r}, want {want.reshape(-1)[i].item()!r}, "
                             f"bound {tol.expand_as(want).reshape(-1)[i].item():.3g}")


def check_bf16(got, want, tol, label):
    check_close(got, want, BF16 * want.abs() + 1.01 * tol + 2.0 ** -134, label)


def check_cast(q, scale_inv, want, tol, fmt, scaling, label, scale=None):
    """An FP8 output (finite values): its scales by the rule, from a maximum
    that is off by at most the values' bound, and its values."""
    tol = tol.expand_as(want)
    v = q.cpu().view(FP8[fmt]).double()
    if scaling == 0:
        x = (want * scale).clamp(-FMAX[fmt], FMAX[fmt])
        t = tol * scale + 2 * U * x.abs()
        check_close(v, x, HALF[fmt] * x.abs() + TINY[fmt] + 1.1 * t, label)
        return
    b = 128 if scaling == 1 else 32
    r, c = want.shape
    a, ta = tiles(want.abs(), b).amax(2), tiles(tol, b).amax(2)
    s = scale_inv.cpu().view(r, -1)
    if scaling == 1:
        s = s.double()
        rule = torch.where(a == 0, torch.ones_like(a), a / FMAX[fmt])
        check_close(s, rule, (ta + 4 * U * a) / FMAX[fmt] + 2.0 ** -149, label + " scales")
    else:
        def byte(m):
            e = torch.ceil(torch.log2(m.clamp(min=2.0 ** -160) / FMAX[fmt]) - 2.0 ** -40)
            return torch.where(m == 0, torch.full_like(m, 127), e.clamp(-127, 127) + 127)
        lo, hi = byte((a - ta - 4 * U * a).clamp(min=0)), byte(a + ta + 4 * U * a)
        got = s.double()
        lo = torch.where((a == 0) & (ta == 0), torch.full_like(lo, 127), lo)
        near0 = (a > 0) & (a <= ta)          # the kernel may see 0 there
        assert bool((((got >= lo) & (got <= hi)) | (near0 & (got == 127))).all()), label + " E8M0"
        s = torch.exp2(got - 127)
    sc = s.repeat_interleave(b, 1)[:, :c]
    t = HALF[fmt] * want.abs() + TINY[fmt] * sc + 1.1 * tol + 8 * U * want.abs()
    check_close(v * sc, want, t, label)


# ------------------------------------------------------------ sorting
def sort_choices(expert, experts, pad, rows):
    """(offsets, counts, pos, src) by a loop over the choices."""
    flat = expert.reshape(-1).tolist()
    counts = [0] * experts
    for e in flat:
        if 0 <= e < experts:
            counts[e] += 1
    offsets = [0]
    for c in counts:
        offsets.append(offsets[-1] + -(-c // pad) * pad)
    at, pos, src = list(offsets), [-1] * len(flat), [-1] * rows
    for i, e in enumerate(flat):
        if 0 <= e < experts:
            pos[i], src[at[e]] = at[e], i
            at[e] += 1
    i32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return i32(offsets), i32(counts), i32(pos).view(expert.shape), i32(src)
