"""Differential attention and the rotary on the GPU where they can go wrong: weights nearly one-hot."""
import math

import pytest

from test_gpu_diff import _lib, _t, check, run  # noqa: F401  (_lib: the fixture that builds)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------- rows with one dominating weight
def shared_mean(B, H, N, d, seed):
    """Keys of each map with a shared mean of norm 40, each query half an earlier key and noise: most
    rows give one key most of the weight."""
    torch = _t()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    m = r(1, 2 * H, 1, d)
    K = 40.0 * m / m.norm(dim=-1, keepdim=True) + r(B, 2 * H, N, d)
    i = torch.arange(N, device="cuda")
    at = (torch.rand(B, 2 * H, N, generator=gen, device="cuda") * i.clamp(min=1)).long().minimum((i - 1).clamp(min=0))
    Q = 0.5 * torch.gather(K, 2, at[..., None].expand_as(K)) + 0.5 * r(B, 2 * H, N, d)
    V, dO = r(B, H, N, 2 * d), r(B, H, N, 2 * d)
    return Q.bfloat16(), K.bfloat16(), V.bfloat16(), torch.linspace(0.2, 0.8, H, device="cuda"), dO.bfloat16()


def heads(x, b, h):
    Q, K, V, lam, dO = x
    return (Q[b:b + 1, 2 * h:2 * h + 2], K[b:b + 1, 2 * h:2 * h + 2], V[b:b + 1, h:h + 1], lam[h:h + 1], dO[b:b + 1, h:h + 1])


@pytest.mark.parametrize("seed,N", [(0, 2048), (1, 1500)])
def test_keys_with_a_shared_mean(seed, N):
    """Every output within its elementwise bound, and dQ within 2e-2 of 64-bit values, this library's
    bound for bf16 outputs on such keys."""
    import diff_reference as R
    torch = _t()
    x = shared_mean(2, 4, N, 64, seed)
    got = run(x)
    vis = R.visible(N, "causal", device="cuda")
    err = size = 0.0
    for b in range(2):
        for h in range(4):
            want = R.with_bounds(*heads(x, b, h), 1, vis)
            mine = {k: got[k][b:b + 1, h:h + 1] for k in ("O", "O2", "dV")}
            mine.update({k: got[k][b:b + 1, 2 * h:2 * h + 2] for k in ("lse", "dQ", "dK")})
            check(mine, want, f"{b} {h}")
            err += (mine["dQ"].double() - want["dQ"][0]).square().sum().item()
            size += want["dQ"][0].square().sum().item()
    assert math.sqrt(err / size) <= 2e-2


def test_a_dominating_weight_is_not_rounded():
    """A weight above a fifth of its row's: its P was past a quarter of the row's sum before it, so it is
    1 exactly and the other weights alone are rounded."""
    import diff_reference as R
    torch = _t()
    N = 1500
    x = shared_mean(1, 2, N, 64, 2)
    got = run(x)["O2"].double()
    vis = R.visible(N, "causal", device="cuda")
    _, want, _, A = R.forward(*x[:4], 1, vis)
    A, v = A[:, :, 1], x[2].double()
    top, at = A.max(-1)
    rest = A.scatter(-1, at[..., None], 0.0)
    tol = 2.0 ** -8 * (rest @ v.abs()) + 1e-5 * (A @ v.abs()) + 2.0 ** -8 * want.abs()
    over = ((got - want).abs() - tol).amax(-1)[top > 0.2]
    assert over.numel() > 1000 and over.max().item() <= 0
