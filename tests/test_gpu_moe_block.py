"""examples/moe_block.py against the same block in 32-bit torch operations.

Each 8-bit rounding of a tensor is off by at most 2^-4 of a value (E4M3's
half step; half of that is its root mean square, and a block's values far
below its largest are off by less than the norm notices).  The roundings that
a result passes through are independent, so its relative distance in the
Frobenius norm is bounded by 2^-4 times the root of their number:
    out       n, W1, a, W2                                                 4
    dweight   as out                                                       4
    dW2       a's three (n, W1, the checkpoint of h), a, dy                5
    dh        n, W1, the checkpoint of h, dy, W2                           5
    dW1       dh's five, dh, n                                             7
    dbeta     dh's five, dh, W1                                            7
    dgamma    as dbeta, and the checkpoint of the normalised rows          8
    dx        as dgamma; it also holds dout itself, which is exact
BF16's roundings between the steps, sixteen times finer, are covered by the
margin between a rounding's root mean square and its bound."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "moe_block.py")
ROUNDINGS = dict(weight=4, w2=5, w1=7, beta=7, gamma=8, x=8)


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("moe_block", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,width,hidden,experts,k", [(200, 256, 128, 4, 2), (7, 128, 384, 16, 3),
                                                           (300, 512, 256, 3, 1)])
def test_moe_block(example, tokens, width, hidden, experts, k):
    block, x, expert, weight, dout = example.make(tokens, width, hidden, experts, k, seed=tokens)
    expert[::11] = -1                            # tokens that no expert takes
    out = block.forward(x, expert, weight)
    grads = block.backward(dout)
    want, want_grads = example.reference(block, x, expert, weight, dout)
    assert torch.equal(out[::11], x[::11])
    assert not grads["weight"][::11].any()
    assert example.relative(out - x, want - x.float()) <= 2 ** -4 * math.sqrt(4)
    for name, n in ROUNDINGS.items():
        got, ref = grads[name], want_grads[name]
        if name == "x":
            got, ref = got.float() - dout.float(), ref - dout.float()
        assert example.relative(got, ref) <= 2 ** -4 * math.sqrt(n), name
