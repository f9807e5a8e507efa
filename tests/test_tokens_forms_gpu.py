"""Attention through the instances and forms that a case reaches only at some
size, bias or cap, against the 64-bit form (token_util's bounds)."""
import pytest
import torch

from test_tokens_gpu import TYPES, _check_attention

pytestmark = pytest.mark.gpu


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
