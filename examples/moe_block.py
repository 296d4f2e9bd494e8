"""One training step of a mixture-of-experts block under MXFP8, with the row
operators around the FP8 GEMMs:

    n = layer norm(x)                          8-bit checkpoint of the normalised rows
    n sorted by expert                         MX operand and BF16 copy
    h = n W1[e]^T, a = silu(h_gate) h_up       MX operand, 8-bit checkpoint of h
    y = a W2[e]^T
    out = x + sum_j weight[t][j] y[choice j]

and the gradients of x, gamma, beta, the routing weights, W1 and W2.  Between
the passes it keeps the two 8-bit checkpoints, the sorted BF16 rows and the
experts' outputs; the activation's output is computed again from h.

    python examples/moe_block.py [--tokens T] [--width C] [--hidden H] [--experts E] [--k K]

prints the step's time and how far the results are from the same block in
32-bit torch operations (relative, in the Frobenius norm).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from scaled_fp8_gemm_amd import fp8sg as F  # noqa: E402

PAD = 128          # rows of an expert's segment are a multiple of it


def _empty(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _mx_pair(x):
    """x [rows][cols] as MX operands along its rows and along its columns."""
    r, c = x.shape
    q, s = _empty(torch.uint8, r, c), _empty(torch.uint8, r, c // 32)
    qT, sT = _empty(torch.uint8, c, r), _empty(torch.uint8, c, r // 32)
    F.fp8_quantize_mx_t(x, F.E4M3, q, s, qT, sT)
    return (F.operand(q, F.E4M3, F.SCALE_MX_1x32, s), F.operand(qT, F.E4M3, F.SCALE_MX_1x32, sT))


class MoeBlock:
    """w1: [experts][2 hidden][width] (gate rows, then up rows), w2:
    [experts][width][hidden], gamma and beta: [width]; all BF16."""

    def __init__(self, w1, w2, gamma, beta, eps=1e-5):
        self.w1, self.w2, self.gamma, self.beta, self.eps = w1, w2, gamma, beta, eps
        self.experts, self.width, self.hidden = w2.shape

    def forward(self, x, expert, weight):
        """x [tokens][width] BF16; expert, weight [tokens][k] (int32, FP32)."""
        (tokens, c), k, h = x.shape, expert.shape[1], self.hidden
        self.w1q = [_mx_pair(w) for w in self.w1]
        self.w2q = [_mx_pair(w) for w in self.w2]
        self.x, self.weight = x, weight
        self.rstd, mean = _empty(torch.float32, tokens), _empty(torch.float32, tokens)
        self.xhat, self.xhat_s = (_empty(torch.uint8, tokens, c),
                                  _empty(torch.float32, tokens, -(-c // 128)))
        n = torch.empty_like(x)
        F.fp8_layernorm_fwd(x, self.gamma, self.beta, self.eps, n, mean, self.rstd,
                            xhat=F.cast_out(self.xhat, F.E4M3, F.SCALE_BLOCK_1x128, self.xhat_s))
        rows = F.moe_rows(tokens * k, self.experts, PAD)
        self.offsets, counts = (_empty(torch.int32, self.experts + 1),
                                _empty(torch.int32, self.experts))
        self.pos, self.src = _empty(torch.int32, tokens, k), _empty(torch.int32, rows)
        F.fp8_moe_sort(expert, self.experts, PAD, self.offsets, counts, self.pos, self.src)
        self.xs = _empty(torch.bfloat16, rows, c)
        xq, xq_s = _empty(torch.uint8, rows, c), _empty(torch.uint8, rows, c // 32)
        F.fp8_moe_dispatch(n, self.pos, self.src, self.offsets, self.xs,
                           xq=F.cast_out(xq, F.E4M3, F.SCALE_MX_1x32, xq_s))
        # the GEMMs are launched per expert: their sizes are needed here
        at = self.offsets.tolist()
        self.segments = [(e, at[e], at[e + 1]) for e in range(self.experts) if at[e + 1] > at[e]]
        self.used = at[-1]
        hs = _empty(torch.bfloat16, self.used, 2 * h)
        for e, a, b in self.segments:
            F.fp8_gemm_fprop(F.operand(xq[a:b], F.E4M3, F.SCALE_MX_1x32, xq_s[a:b]),
                             self.w1q[e][0], b - a, 2 * h, c, hs[a:b])
        act, act_s = _empty(torch.uint8, self.used, h), _empty(torch.uint8, self.used, h // 32)
        self.h, self.h_s = (_empty(torch.uint8, self.used, 2 * h),
                            _empty(torch.float32, self.used * 2, -(-h // 128)))
        F.fp8_act_fwd(hs, F.ACT_SILU, True, None,
                      yq=F.cast_out(act, F.E4M3, F.SCALE_MX_1x32, act_s),
                      ckpt=F.cast_out(self.h, F.E4M3, F.SCALE_BLOCK_1x128, self.h_s))
        self.ys = _empty(torch.bfloat16, rows, c)
        for e, a, b in self.segments:
            F.fp8_gemm_fprop(F.operand(act[a:b], F.E4M3, F.SCALE_MX_1x32, act_s[a:b]),
                             self.w2q[e][0], b - a, c, h, self.ys[a:b])
        y = torch.empty_like(x)
        F.fp8_moe_combine(self.ys, self.pos, weight, y)
        return x + y

    def backward(self, dout):
        """Gradients of x, gamma, beta, weight, w1 and w2."""
        c, h = self.width, self.hidden
        dys, dweight = torch.empty_like(self.ys), torch.empty_like(self.weight)
        F.fp8_moe_combine_bwd(dout, self.ys, self.weight, self.pos, self.src, self.offsets, dys,
                              dweight)
        dw1, dw2 = torch.zeros_like(self.w1), torch.zeros_like(self.w2)
        da = _empty(torch.bfloat16, self.used, h)
        dyT = {}
        for e, a, b in self.segments:
            dy, dyT[e] = _mx_pair(dys[a:b])
            F.fp8_gemm_dgrad(dy, self.w2q[e][1], b - a, c, h, da[a:b])
        dh, act = _empty(torch.bfloat16, self.used, 2 * h), torch.empty_like(da)
        F.fp8_act_bwd(da, F.operand(self.h, F.E4M3, F.SCALE_BLOCK_1x128, self.h_s), F.ACT_SILU,
                      True, dh, y=act)
        dxs = torch.empty_like(self.xs)
        for e, a, b in self.segments:
            F.fp8_gemm_wgrad(dyT[e], _mx_pair(act[a:b])[1], b - a, c, h, dw2[e])
            dhq, dhT = _mx_pair(dh[a:b])
            F.fp8_gemm_dgrad(dhq, self.w1q[e][1], b - a, 2 * h, c, dxs[a:b])
            F.fp8_gemm_wgrad(dhT, _mx_pair(self.xs[a:b])[1], b - a, 2 * h, c, dw1[e])
        dn = torch.empty_like(self.x)
        F.fp8_moe_combine(dxs, self.pos, None, dn)      # the gradient of the dispatch
        dx = torch.empty_like(self.x)
        dgamma, dbeta = _empty(torch.float32, c), _empty(torch.float32, c)
        F.fp8_layernorm_bwd(dn, None, None, self.rstd, self.gamma, dx, dgamma, dbeta,
                            xhat=F.operand(self.xhat, F.E4M3, F.SCALE_BLOCK_1x128, self.xhat_s))
        return dict(x=dout + dx, gamma=dgamma, beta=dbeta, weight=dweight, w1=dw1, w2=dw2)


def reference(block, x, expert, weight, dout):
    """The same block and its gradients in 32-bit torch operations."""
    leaf = {k: v.detach().float().requires_grad_() for k, v in
            dict(x=x, gamma=block.gamma, beta=block.beta, weight=weight, w1=block.w1,
                 w2=block.w2).items()}
    x32 = leaf["x"]
    d = x32 - x32.mean(1, keepdim=True)
    n = d / torch.sqrt((d * d).mean(1, keepdim=True) + block.eps) * leaf["gamma"] + leaf["beta"]
    out = x32
    for e in range(block.experts):
        t, j = torch.nonzero(expert == e, as_tuple=True)
        hh = n[t] @ leaf["w1"][e].t()
        gate, up = hh[:, :block.hidden], hh[:, block.hidden:]
        y = (gate / (1 + torch.exp(-gate)) * up) @ leaf["w2"][e].t()
        out = out.index_add(0, t, y * leaf["weight"][t, j, None])
    out.backward(dout.float())
    return out.detach(), {k: v.grad for k, v in leaf.items()}


def make(tokens, width, hidden, experts, k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()
    block = MoeBlock(normal(experts, 2 * hidden, width, scale=width ** -0.5),
                     normal(experts, width, hidden, scale=hidden ** -0.5),
                     1 + normal(width, scale=0.1), normal(width, scale=0.1))
    x, dout = normal(tokens, width), normal(tokens, width, scale=1e-2)
    score, expert = torch.topk(torch.randn((tokens, experts), generator=g, device="cuda"), k)
    return block, x, expert.int().contiguous(), torch.softmax(score, 1).contiguous(), dout


def relative(a, b):
    return ((a.float() - b).norm() / b.norm()).item()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 2048), ("width", 4096), ("hidden", 2048), ("experts", 8),
                        ("k", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    block, x, expert, weight, dout = make(a.tokens, a.width, a.hidden, a.experts, a.k)
    out = block.forward(x, expert, weight)
    grads = block.backward(dout)
    want, want_grads = reference(block, x, expert, weight, dout)
    print("out %.3f" % relative(out - x, want - x.float()),
          " ".join("d%s %.3f" % (k, relative(grads[k], want_grads[k])) for k in want_grads))
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        block.forward(x, expert, weight)
        block.backward(dout)
    end.record()
    torch.cuda.synchronize()
    print("%.3f ms a step" % (start.elapsed_time(end) / a.steps))


if __name__ == "__main__":
    main()
