"""The 64-bit reference of differential attention pinned on the CPU: its gradients against
autograd and differences, its decomposition into two plain attentions, the rotary's inverse."""
import math

import numpy as np
import pytest
import torch

import diff_reference as R
import oracle


def make(B=1, H=2, g=1, N=9, d=4, seed=0, dtype=torch.float64):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64).to(dtype)  # noqa: E731
    return (r(B, 2 * H, N, d), r(B, 2 * H // g, N, d), r(B, H // g, N, 2 * d), torch.tensor([0.7, -0.3, 0.0, 0.5][:H]).double(),
            r(B, H, N, 2 * d))


@pytest.mark.parametrize("mask,window,docs", [("full", 0, False), ("causal", 0, False), ("causal", 3, False),
                                              ("causal", 1, False), ("causal", 0, True)])
@pytest.mark.parametrize("g", [1, 2])
def test_gradients_match_autograd(mask, window, docs, g):
    Q, K, V, lam, dO = make(B=2, H=2, g=g)
    seg = torch.tensor([[0, 0, 0, 1, 2, 2, 2, 2, 3], [4, 4, 4, 4, 4, 4, 4, 4, 4]]) if docs else None
    vis = R.visible(9, mask, window, seg)
    x = [t.clone().requires_grad_() for t in (Q, K, V, lam)]
    O, O2, lse, _ = R.forward(*x, g, vis)
    want = torch.autograd.grad((O * dO).sum(), x)
    got = R.with_bounds(Q, K, V, lam, dO, g, vis)
    for name, w in zip(("dQ", "dK", "dV", "dlam"), want):
        assert torch.allclose(got[name][0], w, rtol=1e-11, atol=1e-12), name
    h = 1e-5  # differences
    for k, name in enumerate(("dQ", "dK", "dV", "dlam")):
        u = torch.randn(x[k].shape, dtype=torch.float64, generator=torch.Generator().manual_seed(k))
        f = [(R.forward(*[t + sgn * h * u if i == k else t for i, t in enumerate((Q, K, V, lam))], g, vis)[0] * dO).sum()
             for sgn in (1, -1)]
        assert abs((f[0] - f[1]) / (2 * h) - (got[name][0] * u).sum()) <= 1e-8 * (1 + abs(f[0]))


def test_is_the_difference_of_two_attentions():
    Q, K, V, lam, _ = make(N=7)
    O, O2, lse, _ = R.forward(Q, K, V, lam, 1, R.visible(7, "causal"))
    for h in range(2):
        for c in range(2):  # each half of the value head is a plain value head
            v = V[0, h, :, 4 * c:4 * c + 4].numpy()
            o = [oracle.forward(Q[0, 2 * h + m].numpy(), K[0, 2 * h + m].numpy(), v) for m in range(2)]
            assert np.allclose(O[0, h, :, 4 * c:4 * c + 4].numpy(), o[0][0] - lam[h].item() * o[1][0], atol=1e-12)
            assert np.allclose(O2[0, h, :, 4 * c:4 * c + 4].numpy(), o[1][0], atol=1e-12)
            for m in range(2):
                assert np.allclose(lse[0, 2 * h + m].numpy(), o[m][1], atol=1e-12)


@pytest.mark.parametrize("paired", ["half", "neighbour"])
def test_rotary_turns_back_and_keeps_relative_positions(paired):
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(1, 1, 6, 8, generator=gen, dtype=torch.float64)
    pos = torch.arange(6).view(1, 1, 6)
    freq, axis = torch.tensor([1.0, 0.3, 0.01, 2.0]), torch.tensor([0, 0, -1, 0])
    y = R.rope(x, pos, freq, axis, paired)
    assert torch.allclose(R.rope(y, pos, freq, axis, paired, inverse=True), x, atol=1e-13)
    assert torch.allclose(y.norm(dim=-1), x.norm(dim=-1))
    shifted = R.rope(x, pos + 17, freq, axis, paired)
    assert torch.allclose(y @ y.transpose(-1, -2), shifted @ shifted.transpose(-1, -2), atol=1e-12)
    i = 2 if paired == "half" else 4  # pair 2 is copied
    assert torch.equal(y[..., i], x[..., i])
    assert math.isclose(float(R.rope(torch.tensor([[[[1.0, 0, 0, 0, 0, 0, 0, 0]]]]), torch.tensor([[[1]]]), freq, axis,
                                     paired)[0, 0, 0, 0]), math.cos(1.0))
