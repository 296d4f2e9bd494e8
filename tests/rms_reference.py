"""Root-mean-square norm and 4-bit blocks in 64 bits, elementary torch
operations only, with the bounds that the FP32 kernels are held to
(rowop_reference has the units and the checks)."""
import torch

from tests.rowop_reference import U

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ------------------------------------------------------------ RMS norm
def stream(x, delta):
    """The residual stream as it is stored: one FP32 sum, rounded to x's type."""
    return x if delta is None else (x.float() + delta.float()).to(x.dtype)


def rms_fwd(h, gamma, eps):
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    xhat = h * rstd[:, None]
    return rstd, xhat, xhat * gamma


def rms_fwd_bounds(rstd, xhat, y):
    """A square is rounded once and passes at most 8 + 4 additions in its
    thread, 6 in its wave and 16 over the waves: 35 U of the sum of positive
    terms, half of it in the root; the mean, eps, root and reciprocal add less
    than 2 U each.  xhat and y round once more each."""
    rel = 26 * U
    return rel * rstd, (rel + U) * xhat.abs(), (rel + 2 * U) * y.abs()


def rms_bwd(dy, xhat, rstd, gamma, dres):
    g = dy * gamma
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(1, keepdim=True))
    return (dx if dres is None else dx + dres), (dy * xhat).sum(0)


def rms_bwd_bounds(dy, xhat, t_xhat, rstd, gamma, dres):
    """t_xhat: how far the kernel's xhat may be off.  The row's sum passes at
    most 70 roundings (as layer norm's); dx takes 6 more of each term and one
    of the sum with dres; a column's sum is added up row by row."""
    g = (dy * gamma).abs()
    xa = xhat.abs() + t_xhat
    t_c = 72 * U * (g * xa).mean(1, keepdim=True) + (g * t_xhat).mean(1, keepdim=True)
    c = (dy * gamma * xhat).mean(1, keepdim=True).abs()
    t_dx = rstd[:, None] * (6 * U * (g + xa * c) + xa * t_c + t_xhat * c)
    if dres is not None:
        t_dx = t_dx + U * dres.abs() + U * rstd[:, None] * (g + xa * c)
    t_dg = (dy.shape[0] + 80) * U * (dy.abs() * xa).sum(0) + (dy.abs() * t_xhat).sum(0)
    return t_dx, t_dg


# ------------------------------------------------------------ 4-bit blocks
def mx4(x):
    """(codes [r][c], bytes [r][c / 32]) of BF16 or FP64 x, by the rule."""
    r, c = x.shape
    t = x.double().view(r, c // 32, 32)
    big = t.abs().amax(2)                               # NaN stays
    bad = ~torch.isfinite(t).all(2)
    m, e = torch.frexp(torch.where(bad, 1.0, big))      # big = m 2^e, m in [0.5, 1)
    e = torch.where(m <= 0.75, e - 3, e - 2).clamp(-127, 127)
    e = torch.where(big == 0, 0, e)
    a = (t.abs() * torch.exp2(-e.double())[:, :, None])
    mids = torch.tensor([(p + q) / 2 for p, q in zip(E2M1, E2M1[1:])], dtype=torch.float64)
    odd = torch.arange(7) % 2 == 1                      # a tie goes up from an odd code
    a = a[..., None]
    code = ((a > mids) | ((a == mids) & odd)).sum(-1)
    code = torch.where(torch.signbit(t), code + 8, code)
    code = torch.where(bad[:, :, None], 0, code).view(r, c)
    return code, torch.where(bad, 255, e + 127)


def pack(code):
    return (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)


def unpack(q):
    return torch.stack([q.long() % 16, q.long() // 16], -1).view(q.shape[0], 2 * q.shape[1])


def mx4_values(q, byte):
    """Packed codes and scale bytes -> FP64 values, NaN under byte 255."""
    v = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64)[unpack(q.cpu())]
    f = torch.exp2(byte.cpu().double() - 127)
    f = torch.where(byte.cpu() == 255, float("nan"), f)
    return v * f.repeat_interleave(32, 1)
