"""The bound that the corrected delta's tests use can fail: on the CPU, with
the kernels' roundings, it holds with the correction and not without it."""
import pytest
import torch

import delta_util as du
import token_util as tu


def _worst(sign, dtype, dim, softcap, slope, causal):
    gen = torch.Generator().manual_seed(dim)
    n = 60
    q, k, v, do = (t[:, 0].double() for t in du.dominated(gen, [n], 1, 1, dim, dtype, "cpu"))
    seen, away = tu.seen_and_away(n, n, causal, 0, "cpu")
    scale = tu.sqrt_scale(dim)
    dq, dk, r = du.as_rounded(q, k, v, do, scale, softcap, slope, seen, away, dtype, sign)
    eq, ek = du.bounds(r, q, k, v, do, scale, dtype)
    ratio = lambda got, want, e: float(((got - want).abs() /
                                        (e + tu.U[dtype] * want.abs() + tu.LEAST[dtype])).max())
    return ratio(dq, r["dq"], eq), ratio(dk, r["dk"], ek)


CASES = [(dtype, dim, softcap, slope, causal)
         for dtype in (torch.bfloat16, torch.float16) for dim in (64, 128)
         for softcap, slope, causal in ((0.0, 0.0, False), (0.0, 0.01, True), (30.0, 0.01, True))]


@pytest.mark.parametrize("case", CASES, ids=range(len(CASES)))
def test_bound_holds_with_the_correction_only(case):
    dq, dk = _worst(1, *case)
    assert dq <= 1.0 and dk <= 1.0, (dq, dk)
    for sign in (0, -1):
        dq, dk = _worst(sign, *case)
        assert dq > 1.0 and dk > 1.0, (sign, dq, dk)
    dq, dk = _worst("half", *case)
    assert dq > 1.0 and dk <= 1.0, (dq, dk)
