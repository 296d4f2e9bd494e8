"""examples/moe_block.py step by step: every row operator's call of a forward
and a backward pass, recorded with the tensors that it was given, against its
formula in 64 bits under the operator's own bounds, and every step's input
against the step before.  (The block's end-to-end distance from 32-bit
operations is a few percent, all of it 8-bit rounding, in which a missing term
of layer norm's gradient would hide.)"""
import math

import pytest
import torch

from tests import rowop_reference as R
from tests.test_gpu_moe_block import example  # noqa: F401

pytestmark = pytest.mark.gpu

NAMES = ["fp8_layernorm_fwd", "fp8_moe_sort", "fp8_moe_dispatch", "fp8_act_fwd",
         "fp8_moe_combine", "fp8_moe_combine_bwd", "fp8_act_bwd", "fp8_layernorm_bwd"]
# a GEMM's output from BF16 tensors through two 8-bit roundings of at most 2^-4
# of a value each, and its own rounding
TWO = 2.0 ** -4 * math.sqrt(2)


def relative(a, b):
    return ((a.double() - b).norm() / b.norm()).item()


@pytest.mark.parametrize("tokens,width,hidden,experts,k", [(200, 256, 128, 4, 2), (7, 128, 384, 16, 3),
                                                           (300, 512, 256, 3, 1)])
def test_steps(example, monkeypatch, tokens, width, hidden, experts, k):  # noqa: F811
    F, calls = example.F, {}

    def record(name):
        inner = getattr(F, name)

        def call(*args, **kw):
            inner(*args, **kw)
            keep = [a.clone() if isinstance(a, torch.Tensor) else a for a in args]
            calls.setdefault(name, []).append((keep, kw))
        monkeypatch.setattr(F, name, call)
    for name in NAMES:
        record(name)
    block, x, expert, weight, dout = example.make(tokens, width, hidden, experts, k, seed=tokens)
    expert[::11] = -1
    out = block.forward(x, expert, weight)
    grads = block.backward(dout)
    one = {n: c[0] for n, c in calls.items()}
    pos, src = block.pos.cpu().long(), block.src.cpu().long()
    live, real = pos >= 0, src >= 0
    token = torch.where(real, src // k, 0)
    w = weight.cpu().double()

    # ---- forward
    n, mean, rstd = (one["fp8_layernorm_fwd"][0][i].cpu() for i in (4, 5, 6))
    gd, bd, xd = block.gamma.cpu().double(), block.beta.cpu().double(), x.cpu().double()
    m, r, xhat, y = R.ln_fwd(xd, gd, bd, block.eps)
    tm, tr, th, ty = R.ln_fwd_bounds(xd, gd, bd, m, r, xhat)
    R.check_close(mean, m, tm + R.U * m.abs(), "mean")
    R.check_close(rstd, r, tr, "rstd")
    R.check_bf16(n, y, ty, "n")
    R.check_cast(block.xhat, block.xhat_s, xhat, th, 0, 1, "checkpoint of xhat")
    rows = block.src.numel()
    for got, want in zip((block.offsets, block.pos, block.src),
                         [R.sort_choices(expert.cpu(), experts, example.PAD, rows)[i]
                          for i in (0, 2, 3)]):
        assert torch.equal(got.cpu(), want)
    used = block.used
    want = torch.where(real[:, None], n.double()[token], 0.0)[:used]
    assert torch.equal(block.xs[:used].cpu().double(), want)
    hs = one["fp8_act_fwd"][0][0].cpu().double()
    w1, w2 = block.w1.cpu().double(), block.w2.cpu().double()
    for e, a, b in block.segments:
        assert relative(hs[a:b], want[a:b] @ w1[e].t()) <= TWO
    R.check_cast(block.h.view(used * 2, hidden), block.h_s, hs.view(used * 2, hidden),
                 torch.zeros(1, dtype=torch.float64), 0, 1, "checkpoint of h")
    p, _ = R.act_parts(2, hs[:, :hidden])
    a_out = hs[:, :hidden] * p * hs[:, hidden:]
    ys = block.ys.cpu().double()
    for e, a, b in block.segments:
        assert relative(ys[a:b], a_out[a:b] @ w2[e].t()) <= TWO
    comb = one["fp8_moe_combine"][0]
    picked = torch.where(live[:, :, None], ys[pos.clamp(min=0)], 0.0)
    want = (picked * w[:, :, None]).sum(1)
    mag = (picked * w[:, :, None]).abs().sum(1)
    R.check_bf16(comb[3], want, (k + 1) * R.U * mag, "y")
    assert torch.equal(out, x + comb[3])

    # ---- backward
    dy = dout.cpu().double()
    cb = one["fp8_moe_combine_bwd"][0]
    at = torch.where(real, src, 0)
    dys = torch.where(real[:, None], w.view(-1)[at][:, None] * dy[token], 0.0)[:used]
    R.check_bf16(cb[6][:used], dys, R.U * dys.abs(), "dys")
    dots = (picked * dy[:, None]).sum(2)
    R.check_close(grads["weight"], dots, (width / 64 + 32) * R.U * (picked * dy[:, None]).abs().sum(2),
                  "dweight")
    ab = one["fp8_act_bwd"][0]
    da, dh = ab[0].cpu().double(), ab[4].cpu().double()
    dys = cb[6].cpu().double()
    for e, a, b in block.segments:
        assert relative(da[a:b], dys[a:b] @ w2[e]) <= TWO
    h = R.held_values(block.h.view(used * 2, hidden), block.h_s, 0).reshape(used, 2 * hidden)
    g, u = h[:, :hidden], h[:, hidden:]
    p, d = R.act_parts(2, g)
    rel, td = R.act_bounds(2, g)
    td = td + 3 * R.U * g.abs()                    # the held value is one product in FP32
    s = g * p
    ts = s.abs() * (rel + 4 * R.U) + 3 * R.U * g.abs()
    R.check_bf16(ab[4][:, :hidden].contiguous(), da * u * d,
                 (da * u).abs() * (td + 4 * R.U * d.abs()), "dgate")
    R.check_bf16(ab[4][:, hidden:].contiguous(), da * s,
                 da.abs() * (ts + 2 * R.U * s.abs()), "dup")
    dxs, dn = (calls["fp8_moe_combine"][1][0][i].cpu().double() for i in (0, 3))
    for e, a, b in block.segments:
        assert relative(dxs[a:b], dh[a:b] @ w1[e]) <= TWO
    picked = torch.where(live[:, :, None], dxs[pos.clamp(min=0)], 0.0)
    R.check_bf16(dn, picked.sum(1), (k + 1) * R.U * picked.abs().sum(1), "dn")
    lb = one["fp8_layernorm_bwd"][0]
    assert torch.equal(lb[0].cpu().double(), dn) and torch.equal(lb[3], block.rstd)
    xhat, r = R.held_values(block.xhat, block.xhat_s, 0), block.rstd.cpu().double()
    wx, wg, wb = R.ln_bwd(dn, xhat, r, gd)
    tx, tg, tb = R.ln_bwd_bounds(dn, xhat, R.U * xhat.abs(), r, gd)
    R.check_bf16(lb[5], wx, tx, "dx")
    R.check_close(grads["gamma"], wg, tg, "dgamma")
    R.check_close(grads["beta"], wb, tb, "dbeta")
    assert torch.equal(grads["x"], dout + lb[5])
    # the weights' gradients, from the recorded steps
    act = one["fp8_act_bwd"][1]["y"].cpu().double()
    for e, a, b in block.segments:
        assert relative(grads["w1"][e].cpu(), dh[a:b].t() @ block.xs[a:b].cpu().double()) <= TWO
        assert relative(grads["w2"][e].cpu(), dys[a:b].t() @ act[a:b]) <= TWO
    # what the end-to-end distance cannot see, these bounds do: without either
    # of its mean terms the gradient is out of them
    gg = dn * gd
    c1, c2 = gg.mean(1, keepdim=True), (gg * xhat).mean(1, keepdim=True)
    for lost in (r[:, None] * c1, r[:, None] * xhat * c2):
        with pytest.raises(AssertionError):
            R.check_bf16(lb[5], wx + lost, tx, "dx")
