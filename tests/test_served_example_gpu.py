"""The example's layer served in 8 bits: products, cache and attention over it with a
shared prompt, run together."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))


def _tokens(ts, prompt, requests, steps, channels):
    gen = torch.Generator(device="cuda").manual_seed(11)
    x = lambda *shape: torch.randn((*shape, channels), generator=gen, device="cuda").to(ts.HALF)
    return x(prompt), x(steps, requests)


# Rounding to one of n levels of a row is off by span / n / sqrt(12), root mean
# square.  Rows of normal numbers span some six standard deviations, so a value kept
# in 8 bits is off by 0.007 of that deviation, and by 0.12 in 4 bits.  A product of 8
# bits by 8 is off by 0.01, three of them and the cache by 0.02.  In 4 bits a score
# (scaled product with a key, capped) is off by 0.12, and a weight by as much of
# itself; weights and values together are off by 0.17 of the attention's output,
# which is one of two terms of a layer's.
@pytest.mark.parametrize("bits,bound", [(8, 0.04), (4, 0.24)])
def test_served_steps_are_near_those_of_16_bits(bits, bound):
    import token_splats as ts
    layer = ts.TokenLayer()
    prompt, requests, steps = 70, 5, 9
    head, x = _tokens(ts, prompt, requests, steps, layer.C)
    served = ts.Served(layer, requests, steps, prompt, bits)
    served.take_prompt(head)
    got = torch.stack([served.step(t) for t in x])
    cache = layer.start(requests, prompt + steps)
    for t in head:
        layer.step(cache, t.expand(requests, -1).contiguous())
    want = torch.stack([layer.step(cache, t) for t in x])
    err = float((got - want).norm() / want.norm())
    assert err < bound, err


def test_a_shared_prompt_is_the_prompt_of_each():
    """Keys in front of all requests, or copied in front of each one's own: the same
    sums in another order, fp32 apart from the roundings of the results."""
    import token_splats as ts
    layer = ts.TokenLayer()
    prompt, requests, steps = 40, 3, 4
    head, x = _tokens(ts, prompt, requests, steps, layer.C)
    shared = ts.Served(layer, requests, steps, prompt)
    shared.take_prompt(head)
    alone = ts.Served(layer, requests, prompt + steps)
    for t in head:
        alone.step(t.expand(requests, -1).contiguous())
    a = torch.stack([shared.step(t) for t in x])
    b = torch.stack([alone.step(t) for t in x])
    # bf16 results that differ by a rounding, 2^-8, now and then; codes that such a
    # difference moves by one are off by 1 / 127 of a row's largest
    assert float((a - b).norm() / b.norm()) < 0.02


def test_a_captured_step():
    """A step as a graph: the same bits as without, for other tokens and lengths."""
    import token_splats as ts
    layer = ts.TokenLayer()
    requests, room, prompt = 4, 6, 33
    head, x = _tokens(ts, prompt, requests, room, layer.C)
    eager, captured = (ts.Served(layer, requests, room, prompt) for _ in range(2))
    for s in (eager, captured):
        s.take_prompt(head)
    token = x[0].clone()
    one = torch.ones(requests, dtype=torch.int32, device="cuda")
    first = torch.arange(requests, dtype=torch.int32, device="cuda")
    k_len, positions = one.clone(), one * prompt
    raster = ts.raster
    docs = raster.documents(first, one, prompt + first * room, k_len, max_q_len=1,
                            max_k_len=room)
    shared = raster.documents(ts._ints([0]), ts._ints([requests]), ts._ints([0]),
                              ts._ints([prompt]), max_q_len=requests, max_k_len=prompt)
    before = captured.state.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        captured._run(token, positions, docs, shared, captured.state)
    torch.cuda.current_stream().wait_stream(side)
    captured.state.copy_(before)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = captured._run(token, positions, docs, shared, captured.state)
    for i in range(room):
        token.copy_(x[i])
        k_len.fill_(i + 1)
        positions.fill_(prompt + i)
        graph.replay()
        torch.cuda.synchronize()
        want = eager._run(x[i], one * (prompt + i), raster.documents(
            first, one, prompt + first * room, one * (i + 1), max_q_len=1, max_k_len=room),
            shared, eager.state)
        assert torch.equal(out, want)
