"""examples/moe_layer.py: RMS norm with the residual's addition, the sort and
dispatch, the products by expert, the 4-bit weights and their gradients, run
together as a layer, against the same layer in 32-bit torch operations.

Each 8-bit rounding of a tensor is off by at most 2^-4 of a value (E4M3's
half step; half of that is its root mean square, and a block's values far
below its largest are off by less than the norm notices).  The roundings that
a result passes through are independent, so its relative distance in the
Frobenius norm is bounded by 2^-4 times the root of their number:
    out       n, W1, a, W2                                                 4
    dweight   as out                                                       4
    dW2       a's three (n, W1, the checkpoint of u), a, dy                5
    du        n, W1, the checkpoint of u, dy, W2                           5
    dW1       du's five, du, n                                             7
    dgamma    du's five, du, W1, the checkpoint of the normalised rows     8
    dx        as dgamma; it also holds dh itself, which BF16 rounds once
With 4-bit weights the reference takes the weights that the 4 bits hold, which
leaves n and a: 2.  BF16's roundings between the steps, sixteen times finer,
are covered by the margin between a rounding's root mean square and its
bound."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "moe_layer.py")
ROUNDINGS = dict(weight=4, w2=5, w1=7, gamma=8, x=8)
SIZES = [(200, 256, 128, 4, 2), (7, 128, 384, 16, 3), (300, 512, 256, 3, 1), (1, 128, 128, 2, 2)]


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_layer", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def within(example, got, want, roundings):
    return example.relative(got, want) <= 2 ** -4 * math.sqrt(roundings)


@pytest.mark.parametrize("tokens,width,hidden,experts,k", SIZES)
def test_training(example, tokens, width, hidden, experts, k):
    layer, x, delta, expert, weight, dh, dout = example.make(tokens, width, hidden, experts, k,
                                                             seed=tokens)
    expert[3::11] = -1                           # tokens that no expert takes
    h, out = layer.forward(x, delta, expert, weight)
    grads = layer.backward(dh, dout)
    _, want, want_grads = example.reference_grads(layer, x, delta, expert, weight, dh, dout)
    assert torch.equal(h, x + delta)
    assert not out[3::11].any() and not grads["weight"][3::11].any()
    assert torch.equal(grads["x"][3::11], dh[3::11])
    assert within(example, out, want, 4)
    for name, n in ROUNDINGS.items():
        got, ref = grads[name], want_grads[name]
        if name == "x":
            got, ref = got.float() - dh.float(), ref - dh.float()
        assert within(example, got, ref, n), name


def test_gradients_against_differences(example):
    """Along its own direction u = g / |g| the slope of the loss is |g|; the
    layer's gradient differs from g by at most the bound above times |g|, so
    its slope does too (Cauchy and Schwarz).  The slope is taken in 64 bits
    over +-1e-4 |v| on either side, whose second-order error is far below."""
    layer, x, delta, expert, weight, dh, dout = example.make(96, 256, 128, 4, 2, seed=5)
    layer.forward(x, delta, expert, weight)
    grads = layer.backward(dh, dout)
    at = dict(x=x, gamma=layer.gamma, weight=weight, w1=layer.w1, w2=layer.w2)
    at = {k: v.double() for k, v in at.items()}

    def loss(**moved):
        v = dict(at, **moved)
        h, out = example.reference(v["w1"], v["w2"], v["gamma"], layer.eps, v["x"],
                                   delta.double(), expert, v["weight"], torch.float64)
        return (h * dh.double()).sum() + (out * dout.double()).sum()
    for name, n in ROUNDINGS.items():
        g = grads[name].double()
        u = g / g.norm()
        step = 1e-4 * at[name].norm()
        slope = (loss(**{name: at[name] + step * u}) - loss(**{name: at[name] - step * u})) / (2 * step)
        # |g_layer - g| <= b |g| and |g| <= |g_layer| / (1 - b)
        b = 2 ** -4 * math.sqrt(n)
        assert abs(slope - g.norm()) <= b / (1 - b) * g.norm(), name


@pytest.mark.parametrize("tokens,width,hidden,experts,k", SIZES)
def test_serving(example, tokens, width, hidden, experts, k):
    layer, x, delta, expert, weight, _, _ = example.make(tokens, width, hidden, experts, k,
                                                         seed=tokens + 1)
    expert[3::11] = -1
    served = example.ServedLayer(layer)
    h, out = served.forward(x, delta, expert, weight)
    _, want = example.reference(*(w.float() for w in served.held()), layer.gamma.float(),
                                layer.eps, x.float(), delta.float(), expert, weight)
    assert torch.equal(h, x + delta) and not out[3::11].any()
    assert within(example, out, want, 2)


@pytest.mark.parametrize("served", [False, True])
def test_graph(example, served):
    """A captured step replayed for other rows, another routing and, with the
    program's own work between, again: every result as the eager step's."""
    sizes = (130, 256, 128, 5, 2)
    layer, x, delta, expert, weight, dh, dout = example.make(*sizes, seed=1)
    if served:
        layer = example.ServedLayer(layer)

    def step(layer=layer):
        res = list(layer.forward(x, delta, expert, weight))
        return res + ([] if served else list(layer.backward(dh, dout).values()))
    graph, held = example.captured(step)
    eager = (example.ServedLayer if served else example.MoeLayer)
    for seed in (1, 2, 3, 2):
        _, *new = example.make(*sizes, seed=seed)
        new[2][seed::7] = -1
        if seed == 3:
            new[2].fill_(4)                      # every choice to one expert
        for a, b in zip((x, delta, expert, weight, dh, dout), new):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        other = eager(layer) if served else eager(layer.w1, layer.w2, layer.gamma)
        for i, (a, b) in enumerate(zip(got, step(other))):
            assert torch.equal(a, b), (seed, i)
