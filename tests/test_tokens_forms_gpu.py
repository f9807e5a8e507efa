"""Attention through every kernel instance and form, against the 64-bit form
(token_util's bounds); the kernels that a case is meant for are looked up in a
trace of its calls, so that a changed rule cannot move it to others unseen."""
import re

import pytest
import torch

import token_util as tu
from test_tokens_gpu import TYPES, _check_attention, _run_attention

pytestmark = pytest.mark.gpu
NAMES = {torch.bfloat16: "Bf16", torch.float16: "F16"}


# caps far above the scores: they leave them as they are, to fp32 accuracy
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("softcap", [65.0, 1e3, 1e5, 1e9, 2.0 ** 100])
@pytest.mark.parametrize("case", [
    ([130, 65, 257, 1], None, 4, 2, 64, dict(causal=True)),
    ([130, 65], None, 3, 1, 128, dict(causal=False, slopes=True)),
    ([1, 1], [900, 300], 8, 2, 96, dict(causal=True)),
    ([130, 165], None, 64, 32, 64, dict(causal=True, prefix=[20, 0])),
    ([130, 165], None, 64, 64, 128, dict(causal=True))], ids=range(5))
def test_attention_large_caps(case, softcap, dtype):
    _check_attention(case[:5] + (dict(case[5], softcap=softcap),), dtype, "rows")


def _kernels_of(case, dtype):
    """Names of the attention kernels that the case launches, without types:
    {"fwd", "join", ...: (elements, mode)}; empty where nothing is traced."""
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA]) as trace:
        _run_attention(case, dtype, "fused")
        torch.cuda.synchronize()
    found = {}
    for e in trace.events():
        m = re.search(r"attention_(\w+)_kernel<gs::(\w+)(?:, (\d+), (\d+))?>", e.name)
        if m:
            assert m[2] == NAMES[dtype]
            found[m[1]] = (int(m[3]), int(m[4])) if m[3] else None
    return found


def _check_kernels(case, dtype, want):
    found = _kernels_of(case, dtype)
    if found:
        assert found == want, (found, want)


# how scores are made, and the number of their kind in the kernels' names
SCORES = [(0, {}), (1, dict(softcap=6.0)), (2, dict(slopes=True)),
          (3, dict(softcap=6.0, slopes=True)), (7, dict(softcap=200.0)),
          (7, dict(softcap=200.0, slopes=True))]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dim", [40, 64, 96, 128])
@pytest.mark.parametrize("mode,scores", SCORES, ids=range(len(SCORES)))
def test_attention_every_instance(mode, scores, dim, dtype):
    """Each way to make scores, by 128 columns and keys a workgroup (many heads)
    and by 32 (few), with a document shorter than a tile of keys, one that ends
    inside a tile, and a prefix."""
    elements = 64 if dim <= 64 else 128
    masks = dict(causal=True, prefix=[0, 90, 3])
    wide = ([150, 129, 31], None, 160, 80, dim, dict(scores, **masks))
    _check_attention(wide, dtype, "fused")
    at = (elements, mode)
    _check_kernels(wide, dtype, {"fwd": at, "dq": at, "dkv": at, "heads": None})
    few = ([150, 129, 31], None, 4, 2, dim, dict(scores, **masks))
    _check_attention(few, dtype, "heads")
    _check_kernels(few, dtype, {"step": at, "dq_few": at, "dkv_few": at, "heads": None})


@pytest.mark.parametrize("scale", [-0.15, 0.0])
@pytest.mark.parametrize("heads", [(4, 2), (160, 80)])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_scales_that_are_not_positive(dim, heads, scale, monkeypatch):
    monkeypatch.setattr(tu, "sqrt_scale", lambda dim: scale)
    for scores in ({}, dict(softcap=5.0)):
        case = ([150, 129, 31], None, *heads, dim, dict(scores, causal=True))
        _check_attention(case, torch.float16, "rows")


FORMS = [
    # documents of more than 2,560 keys in pieces: pieces wholly past a causal
    # column tile's end, and the join of their empty sums
    (([3000], None, 1, 1, 64, dict(causal=True)), {"step", "join", "dq_few", "dkv_few"}),
    (([40, 100], [3000, 2700], 2, 1, 128, dict(causal=True)),
     {"step", "join", "dq_few", "dkv_few", "heads"}),
    (([100, 40], [2600, 3100], 2, 1, 40, dict(causal=True, slopes=True, softcap=9.0)),
     {"step", "join", "dq_few", "dkv_few", "heads"}),
    # many one-token requests: all first pieces before all second ones
    (([1] * 40, [700 + 37 * i for i in range(40)], 16, 8, 64, dict(causal=True)),
     {"step", "join"}),
    (([1] * 40, [1500 - 37 * i for i in range(40)], 16, 8, 128,
      dict(causal=True, slopes=True, softcap=12.0)), {"step", "join"}),
    (([0, 1, 2] * 14, [0, 900, 1300] * 14, 16, 8, 96, dict(causal=True)), {"step", "join"}),
    # enough key tiles that a workgroup adds the query heads itself
    (([3] * 699 + [70], None, 8, 4, 64, dict(causal=True, slopes=True)), {"fwd", "dq", "dkv"}),
    (([2] * 699 + [140], None, 12, 4, 128, dict(causal=True, softcap=7.0)), {"fwd", "dq", "dkv"}),
]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("case,kernels", FORMS, ids=range(len(FORMS)))
def test_attention_forms(case, kernels, dtype):
    _check_attention(case, dtype, "fused")
    found = _kernels_of(case, dtype)
    if found:
        assert kernels <= set(found), found
        assert "fwd" not in kernels or "heads" not in found


@pytest.mark.parametrize("case", [
    ([150, 129, 31], None, 160, 80, 64, dict(causal=True, slopes=True)),
    ([150, 129, 31], None, 160, 80, 128, dict(causal=True, softcap=6.0, slopes=True)),
    ([300, 20], None, 128, 128, 128, dict(causal=False)),
    FORMS[1][0], FORMS[3][0], FORMS[6][0]], ids=range(6))
def test_attention_forms_repeat_bit_for_bit_and_on_another_stream(case):
    a = _run_attention(case, torch.bfloat16, "rows")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = _run_attention(case, torch.bfloat16, "rows")
    side.synchronize()
    for n in ("o", "lse", "dq", "dk", "dv"):
        x, y = a[n], b[n]
        assert ((x == y) | (torch.isnan(x) & torch.isnan(y))).all(), n
