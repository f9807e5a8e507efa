"""The example network end to end: training through the rasterizer lowers the
loss, its gradient agrees with differences, and the one-token form gives what
the whole-document form gives."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def test_training_lowers_the_loss():
    import token_splats
    losses, _ = token_splats.train(steps=40, sizes=(150, 33, 257))
    assert all(x == x for x in losses)
    assert losses[-1] < 0.7 * losses[0], (losses[0], losses[-1])


def test_head_gradient_against_differences():
    """dL/d(head) through the rasterizer along a direction (the head's product
    is fp32, so differences of the rendered loss resolve it)."""
    import token_splats as ts
    data, layer = ts.Scenes([120, 65]), ts.TokenLayer()
    x = data.tokens(layer.C)
    _, dp = data.loss(layer.forward(x, data.positions, data.docs))
    g = layer.backward(dp)["head"]
    direction = g / g.norm()
    base, h = layer.w["head"].clone(), 1e-3
    values = []
    for sign in (1, -1):
        layer.w["head"] = base + sign * h * direction
        values.append(data.loss(layer.forward(x, data.positions, data.docs))[0])
    want, have = (values[0] - values[1]) / (2 * h), float((g * direction).sum())
    # skipped and clamped pairs make the loss uneven at the size of the step
    assert abs(have - want) <= 0.03 * abs(have), (have, want)


def test_steps_equal_the_whole_document():
    import token_splats as ts
    layer = ts.TokenLayer()
    n, requests = 70, 3
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn((requests, n, layer.C), generator=gen, device="cuda").to(ts.HALF)
    docs = ts.raster.documents(ts._ints([i * n for i in range(requests)]),
                               ts._ints([n] * requests), max_q_len=n)
    positions = torch.arange(n, dtype=torch.int32, device="cuda").repeat(requests)
    whole = layer.forward(x.view(-1, layer.C), positions, docs).view(requests, n, -1)
    cache = layer.start(requests, n)
    steps = torch.stack([layer.step(cache, x[:, t].contiguous()) for t in range(n)], 1)
    # a handful of bfloat16 roundings (2^-9 of a value each, root mean square)
    # in a chain: q and k, the weights, o, y, gate and input, the scan's output
    err = float((steps - whole).norm() / whole.norm())
    assert err < 8 * 2.0 ** -9, err
