"""A mixture-of-experts layer between two additions to the residual stream,
for training under MXFP8 and for serving with 4-bit weights:

    h = x + delta, n = RMS norm(h)             8-bit checkpoint of the normalised rows
    n sorted by expert                         MX operand and BF16 copy
    u = n W1[e]^T, a = silu(u_gate) u_up       one product over all experts; MX operand
    y = a W2[e]^T, out = sum_j weight[t][j] y[choice j]

h goes on along the stream and `out` is the next layer's delta.  Where the
experts' segments begin stays on the GPU, so nothing waits for the host and a
step is captured into a graph once and replayed for any routing.

    python examples/moe_layer.py [--tokens T] [--width C] [--hidden H] [--experts E] [--k K]

prints the time of a captured training step and of a captured serving step of
16 tokens, and how far the results are from 32-bit torch operations (relative,
in the Frobenius norm).
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from scaled_fp8_gemm_amd import fp8sg as F  # noqa: E402


def _empty(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _mx_pair(x):
    """x [rows][cols] as MX operands along its rows and along its columns."""
    r, c = x.shape
    q, s = _empty(torch.uint8, r, c), _empty(torch.uint8, r, c // 32)
    qT, sT = _empty(torch.uint8, c, r), _empty(torch.uint8, c, r // 32)
    F.fp8_quantize_mx_t(x, F.E4M3, q, s, qT, sT)
    return (F.operand(q, F.E4M3, F.SCALE_MX_1x32, s), F.operand(qT, F.E4M3, F.SCALE_MX_1x32, sT))


def _mx_weights(w):
    """w [experts][n][k] as MX operands of the products by expert, each
    expert's matrix along its rows and along its columns."""
    e, n, k = w.shape
    q, s = _empty(torch.uint8, e, n, k), _empty(torch.uint8, e, n, k // 32)
    qT, sT = _empty(torch.uint8, e, k, n), _empty(torch.uint8, e, k, n // 32)
    for i in range(e):
        F.fp8_quantize_mx_t(w[i], F.E4M3, q[i], s[i], qT[i], sT[i])
    return (F.operand(q, F.E4M3, F.SCALE_MX_1x32, s), F.operand(qT, F.E4M3, F.SCALE_MX_1x32, sT))


def _mx4_weights(w):
    """w [experts][n][k] in 4 bits, its blocks along its rows."""
    e, n, k = w.shape
    q, s = _empty(torch.uint8, e, n, k // 2), _empty(torch.uint8, e, n, k // 32)
    F.fp8_quantize_mx4(w.view(e * n, k), q, s)
    return F.operand(q, F.FP4_E2M1, F.SCALE_MX_1x32, s)


class MoeLayer:
    """w1: [experts][2 hidden][width] (gate rows, then up rows), w2:
    [experts][width][hidden], gamma [width]; all BF16."""

    PAD = 128      # segments of whole MX blocks, and of 128 rows of the weights' gradients

    def __init__(self, w1, w2, gamma, eps=1e-5):
        self.w1, self.w2, self.gamma, self.eps = w1, w2, gamma, eps
        self.experts, self.width, self.hidden = w2.shape

    def _sorted(self, n, expert, pad, keep):
        """n's rows by expert: the MX operand, and the BF16 copy with `keep`."""
        c, rows = self.width, F.moe_rows(expert.numel(), self.experts, pad)
        self.offsets, counts = (_empty(torch.int32, self.experts + 1),
                                _empty(torch.int32, self.experts))
        self.pos, self.src = torch.empty_like(expert), _empty(torch.int32, rows)
        F.fp8_moe_sort(expert, self.experts, pad, self.offsets, counts, self.pos, self.src)
        self.xs = _empty(torch.bfloat16, rows, c) if keep else None
        q, s = _empty(torch.uint8, rows, c), _empty(torch.uint8, rows, c // 32)
        F.fp8_moe_dispatch(n, self.pos, self.src, self.offsets, self.xs,
                           xq=F.cast_out(q, F.E4M3, F.SCALE_MX_1x32, s))
        return F.operand(q, F.E4M3, F.SCALE_MX_1x32, s), rows

    def _experts(self, xq, rows, w1q, w2q, ckpt):
        """The experts' outputs of the sorted rows."""
        c, h = self.width, self.hidden
        u = _empty(torch.bfloat16, rows, 2 * h)
        F.fp8_gemm_grouped_fprop(xq, w1q, self.offsets, self.experts, rows, 2 * h, c, u)
        q, s = _empty(torch.uint8, rows, h), _empty(torch.uint8, rows, h // 32)
        F.fp8_act_fwd(u, F.ACT_SILU, True, None, yq=F.cast_out(q, F.E4M3, F.SCALE_MX_1x32, s),
                      ckpt=ckpt)
        ys = _empty(torch.bfloat16, rows, c)
        F.fp8_gemm_grouped_fprop(F.operand(q, F.E4M3, F.SCALE_MX_1x32, s), w2q, self.offsets,
                                 self.experts, rows, c, h, ys)
        return ys

    def forward(self, x, delta, expert, weight):
        """x, delta [tokens][width] BF16; expert, weight [tokens][k] (int32,
        FP32): h and the layer's output."""
        tokens, c = x.shape
        self.weight = weight
        self.w1q, self.w2q = _mx_weights(self.w1), _mx_weights(self.w2)
        self.rstd = _empty(torch.float32, tokens)
        self.xhat, self.xhat_s = (_empty(torch.uint8, tokens, c),
                                  _empty(torch.float32, tokens, -(-c // 128)))
        h, n = torch.empty_like(x), torch.empty_like(x)
        F.fp8_rmsnorm_fwd(x, delta, self.gamma, self.eps, h, n, self.rstd,
                          xhat=F.cast_out(self.xhat, F.E4M3, F.SCALE_BLOCK_1x128, self.xhat_s))
        xq, rows = self._sorted(n, expert, self.PAD, True)
        self.u, self.u_s = (_empty(torch.uint8, rows, 2 * self.hidden),
                            _empty(torch.float32, rows * 2, -(-self.hidden // 128)))
        self.ys = self._experts(xq, rows, self.w1q[0], self.w2q[0],
                                F.cast_out(self.u, F.E4M3, F.SCALE_BLOCK_1x128, self.u_s))
        out = torch.empty_like(x)
        F.fp8_moe_combine(self.ys, self.pos, weight, out)
        return h, out

    def backward(self, dh, dout):
        """Gradients of x (and delta: they are the same), gamma, weight, w1
        and w2 from those of h and of the output."""
        (rows, c), h, off, e = self.ys.shape, self.hidden, self.offsets, self.experts
        dys, dweight = torch.empty_like(self.ys), torch.empty_like(self.weight)
        F.fp8_moe_combine_bwd(dout, self.ys, self.weight, self.pos, self.src, off, dys, dweight)
        dy, dyT = _mx_pair(dys)
        da = _empty(torch.bfloat16, rows, h)
        F.fp8_gemm_grouped_dgrad(dy, self.w2q[1], off, e, rows, c, h, da)
        du, act = _empty(torch.bfloat16, rows, 2 * h), torch.empty_like(da)
        F.fp8_act_bwd(da, F.operand(self.u, F.E4M3, F.SCALE_BLOCK_1x128, self.u_s), F.ACT_SILU,
                      True, du, y=act)
        dw1, dw2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        F.fp8_gemm_grouped_wgrad(dyT, _mx_pair(act)[1], off, e, rows, c, h, dw2)
        duq, duT = _mx_pair(du)
        dxs = torch.empty_like(self.ys)
        F.fp8_gemm_grouped_dgrad(duq, self.w1q[1], off, e, rows, 2 * h, c, dxs)
        F.fp8_gemm_grouped_wgrad(duT, _mx_pair(self.xs)[1], off, e, rows, 2 * h, c, dw1)
        dn, dx = torch.empty_like(dout), torch.empty_like(dh)
        F.fp8_moe_combine(dxs, self.pos, None, dn)      # the gradient of the dispatch
        dgamma = _empty(torch.float32, c)
        F.fp8_rmsnorm_bwd(dn, None, self.rstd, self.gamma, dh, dx, dgamma,
                          xhat=F.operand(self.xhat, F.E4M3, F.SCALE_BLOCK_1x128, self.xhat_s))
        return dict(x=dx, gamma=dgamma, weight=dweight, w1=dw1, w2=dw2)


class ServedLayer(MoeLayer):
    """The same layer's forward pass with its weights laid out once in 4 bits;
    nothing is kept for a backward pass."""

    PAD = 16

    def __init__(self, layer):
        super().__init__(layer.w1, layer.w2, layer.gamma, layer.eps)
        self.w1q, self.w2q = _mx4_weights(layer.w1), _mx4_weights(layer.w2)

    def held(self):
        """The weights that the 4 bits hold, in BF16."""
        w1, w2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        for w, o in ((w1, self.w1q), (w2, self.w2q)):
            q, s = o._tensors
            F.fp8_dequantize_mx4(q, s, w.shape[0] * w.shape[1], w.shape[2], w)
        return w1, w2

    def forward(self, x, delta, expert, weight):
        h, n, rstd = torch.empty_like(x), torch.empty_like(x), _empty(torch.float32, x.shape[0])
        F.fp8_rmsnorm_fwd(x, delta, self.gamma, self.eps, h, n, rstd)
        xq, rows = self._sorted(n, expert, self.PAD, False)
        ys, out = self._experts(xq, rows, self.w1q, self.w2q, None), torch.empty_like(x)
        F.fp8_moe_combine(ys, self.pos, weight, out)
        return h, out


def reference(w1, w2, gamma, eps, x, delta, expert, weight, dtype=torch.float32):
    """The layer in torch operations: h and the output."""
    hidden = w2.shape[2]
    h = x + delta
    n = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * gamma
    out = torch.zeros_like(h)
    for e in range(w2.shape[0]):
        t, j = torch.nonzero(expert == e, as_tuple=True)
        u = n[t] @ w1[e].to(dtype).t()
        gate, up = u[:, :hidden], u[:, hidden:]
        y = (gate / (1 + torch.exp(-gate)) * up) @ w2[e].to(dtype).t()
        out = out.index_add(0, t, y * weight[t, j, None])
    return h, out


def reference_grads(layer, x, delta, expert, weight, dh, dout):
    leaf = {k: v.detach().float().requires_grad_() for k, v in
            dict(x=x, gamma=layer.gamma, weight=weight, w1=layer.w1, w2=layer.w2).items()}
    h, out = reference(leaf["w1"], leaf["w2"], leaf["gamma"], layer.eps, leaf["x"], delta.float(),
                       expert, leaf["weight"])
    torch.autograd.backward((h, out), (dh.float(), dout.float()))
    return h.detach(), out.detach(), {k: v.grad for k, v in leaf.items()}


def make(tokens, width, hidden, experts, k, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()
    layer = MoeLayer(normal(experts, 2 * hidden, width, scale=width ** -0.5),
                     normal(experts, width, hidden, scale=hidden ** -0.5),
                     1 + normal(width, scale=0.1))
    x, delta = normal(tokens, width), normal(tokens, width)
    dh, dout = normal(tokens, width, scale=1e-2), normal(tokens, width, scale=1e-2)
    score, expert = torch.topk(torch.randn((tokens, experts), generator=g, device="cuda"), k)
    return (layer, x, delta, expert.int().contiguous(), torch.softmax(score, 1).contiguous(), dh,
            dout)


def captured(call):
    """call() recorded into a graph, after a run on a stream of its own: the
    graph and what the recorded call returned."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    return graph, out


def relative(a, b):
    return ((a.float() - b).norm() / b.norm()).item()


def _timed(graph, steps):
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    start.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return start.elapsed_time(end) / steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 2048), ("width", 4096), ("hidden", 2048), ("experts", 8),
                        ("k", 2)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--steps", type=int, default=10)
    a = ap.parse_args()
    layer, x, delta, expert, weight, dh, dout = make(a.tokens, a.width, a.hidden, a.experts, a.k)
    _, out = layer.forward(x, delta, expert, weight)
    grads = layer.backward(dh, dout)
    _, want, want_grads = reference_grads(layer, x, delta, expert, weight, dh, dout)
    print("out %.3f" % relative(out, want),
          " ".join("d%s %.3f" % (k, relative(grads[k], want_grads[k])) for k in want_grads))
    graph, _ = captured(lambda: (layer.forward(x, delta, expert, weight),
                                 layer.backward(dh, dout)))
    print("%.3f ms a training step" % _timed(graph, a.steps))
    few = [t[:16].contiguous() for t in (x, delta, expert, weight)]
    served = ServedLayer(layer)
    w = [layer.gamma.float()]
    _, out = served.forward(*few)
    f32 = [few[0].float(), few[1].float(), few[2], few[3]]
    _, want = reference(*(t.float() for t in served.held()), *w, layer.eps, *f32)
    graph, _ = captured(lambda: served.forward(*few))
    print("out %.3f, %.3f ms for %d tokens with 4-bit weights"
          % (relative(out, want), _timed(graph, a.steps), few[0].shape[0]))


if __name__ == "__main__":
    main()
