"""The 64-bit forms that the token operators' kernels are held against,
checked on the CPU: gradients against central differences, the scan's coupled
form against compositing, the rotation's properties."""
import pytest
import torch

import token_util as tu

torch.manual_seed(0)
D = torch.float64


def _directional(fn, tensors, grads, seed, step=1e-5):
    """<gradient, direction> and the central difference along it."""
    gen = torch.Generator().manual_seed(seed)
    for t, g in zip(tensors, grads):
        d = torch.randn(t.shape, generator=gen, dtype=D)
        keep = t.clone()
        t.copy_(keep + step * d)
        hi = float(fn())
        t.copy_(keep - step * d)
        lo = float(fn())
        t.copy_(keep)
        want = (hi - lo) / (2 * step)
        have = float((g * d).sum())
        assert abs(have - want) <= 1e-6 * max(1.0, abs(want)), (have, want)


@pytest.mark.parametrize("softcap", [0.0, 5.0])
@pytest.mark.parametrize("causal,prefix,lq,lk", [(False, 0, 5, 7), (True, 0, 6, 6), (True, 3, 6, 6),
                                                 (True, 0, 7, 4), (True, 2, 7, 4)])
def test_attention_gradient_against_differences(softcap, causal, prefix, lq, lk):
    gen = torch.Generator().manual_seed(lq * 10 + lk)
    q, k, v, w = (torch.randn((n, 8), generator=gen, dtype=D) for n in (lq, lk, lk, lq))
    seen, away = tu.seen_and_away(lq, lk, causal, prefix, "cpu")
    f = lambda: (tu.attention_head(q, k, v, None, 0.4, softcap, 0.3, seen, away)["o"] * w).sum()
    r = tu.attention_head(q, k, v, w, 0.4, softcap, 0.3, seen, away)
    assert (r["o"][r["none"]] == 0).all()
    _directional(f, (q, k, v), (r["dq"], r["dk"], r["dv"]), 3)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_qk_gradient_against_differences(interleaved, norm):
    gen = torch.Generator().manual_seed(4)
    x, dy = (torch.randn((5, 2, 24), generator=gen, dtype=D) for _ in range(2))
    w = 1 + 0.3 * torch.randn(24, generator=gen, dtype=D)
    pos = torch.tensor([0, 1, 7, 900, 60000])
    turn = tu.turn_matrix(pos, torch.rand(8, generator=gen, dtype=D), 24, 16, interleaved, 1.2)
    f = lambda: (tu.qk_forward(x, w if norm else None, turn, 1e-3)[0] * dy).sum()
    dx, _, dw, _ = tu.qk_backward(x, w if norm else None, turn, 1e-3, dy)
    _directional(f, (x, w) if norm else (x,), (dx, dw) if norm else (dx,), 5)


def test_rotation_keeps_lengths_and_depends_on_differences():
    pos = torch.tensor([3, 10])
    freq = torch.tensor([1.0, 0.2, 0.01, 0.003], dtype=D)
    for interleaved in (False, True):
        a = tu.turn_matrix(pos, freq, 8, 8, interleaved, 1.0)
        b = tu.turn_matrix(pos + 1000, freq, 8, 8, interleaved, 1.0)
        assert torch.allclose(a[0] @ a[0].T, torch.eye(8, dtype=D), atol=1e-12)
        assert torch.allclose(a[0].T @ a[1], b[0].T @ b[1], atol=1e-9)


@pytest.mark.parametrize("coupled", [False, True])
def test_scan_gradient_against_differences(coupled):
    gen = torch.Generator().manual_seed(6)
    f, x, dy = (torch.randn((9, 4), generator=gen, dtype=D) for _ in range(3))
    h0, dh = (torch.randn(4, generator=gen, dtype=D) for _ in range(2))

    def loss():
        r = tu.scan_document(f, x, h0, coupled)
        return (r["y"] * dy).sum() + (r["state"] * dh).sum()
    r = tu.scan_document(f, x, h0, coupled, dy, dh)
    _directional(loss, (f, x, h0), (r["df"], r["dx"], r["dstate"]), 7)


def test_coupled_scan_is_back_to_front_compositing():
    gen = torch.Generator().manual_seed(8)
    gate, x = (torch.randn((6, 3), generator=gen, dtype=D) for _ in range(2))
    bg = torch.randn(3, generator=gen, dtype=D)
    alpha = torch.sigmoid(-gate)
    # front to back over the reversed order: C = sum alpha T c + T background
    c, T = torch.zeros(3, dtype=D), torch.ones(3, dtype=D)
    for t in range(5, -1, -1):
        c = c + alpha[t] * T * x[t]
        T = T * (1 - alpha[t])
    assert torch.allclose(tu.scan_document(gate, x, bg, True)["state"], c + T * bg, atol=1e-12)
