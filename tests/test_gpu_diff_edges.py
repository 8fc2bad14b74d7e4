"""Differential attention and the rotary on the GPU where they can go wrong: weights nearly one-hot, infinite
scores, angles of far positions, two streams at once, offsets past 2^31 elements."""
import math
from fractions import Fraction

import pytest

from test_gpu_diff import _lib, _t, check, decode_reference, dt, make, run  # noqa: F401  (_lib: the fixture that builds)

pytestmark = pytest.mark.gpu


# -------------------------------------------------------------- offsets past 2^31 elements
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_last_head_past_2_31_elements(dtype):
    """17 heads of 2^20 tokens: the last head of every tensor begins at 2^31 elements.  Forward, backward,
    a token over the cache and the rotary, which also reads and writes a projection's layout there."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    H, N, d, W = 17, 1 << 20, 64, 40
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(0)

    def big(heads, width):  # the last head's values random, the others' zero
        x = torch.zeros(1, heads, N, width, dtype=dt(dtype), device="cuda")
        x[:, -(heads // H):] = torch.randn(1, heads // H, N, width, generator=gen, device="cuda").to(dt(dtype))
        assert (heads - heads // H) * N * width == 1 << 31
        return x

    Q, K, V, dO = big(2 * H, d), big(2 * H, d), big(H, 2 * d), big(H, 2 * d)
    lam = torch.full((H,), 0.5, device="cuda")
    last = (*(t[:, -(t.shape[1] // H):].contiguous() for t in (Q, K, V)), lam[-1:], dO[:, -1:].contiguous())
    a, b = run((Q, K, V, lam, dO), window=W), run(last, window=W)
    for k in b:
        got = a[k][-1:] if k == "dlam" else a[k][:, -(a[k].shape[1] // H):]
        assert torch.equal(got, b[k]), k
    del a, b, dO
    lens = torch.tensor([N], dtype=torch.int32, device="cuda")
    o = fbd.attn_diff_decode(Q[:, :, -1:].contiguous(), K, V, lam, lens)
    want, tol = decode_reference(last[0][:, :, -1:], last[1], last[2], last[3], lens, 1)
    assert ((o[:, -1:].double() - want).abs() <= tol).all()
    del K, V
    pos = torch.arange(N, device="cuda", dtype=torch.int32)[None]
    freq, axis = torch.rand(d // 2, device="cuda"), torch.zeros(d // 2, dtype=torch.int32, device="cuda")
    turned = fbd.attn_rope(last[0], pos, freq, axis)
    assert torch.equal(fbd.attn_rope(Q, pos, freq, axis)[:, -2:], turned)
    del Q
    # [B, N, heads, d]: the last token begins past 2^31 elements
    proj = torch.zeros(1, N, 2 * H, d, dtype=dt(dtype), device="cuda")
    proj[:, :, -2:] = last[0].transpose(1, 2)
    y = fbd.attn_rope(proj.transpose(1, 2), pos, freq, axis)
    assert torch.equal(y[:, -2:], turned)
    proj.zero_()
    fbd.attn_rope(y, pos, freq, axis, inverse=True, outs=proj.transpose(1, 2))
    assert torch.equal(proj[:, :, -2:].transpose(1, 2), fbd.attn_rope(turned, pos, freq, axis, inverse=True))
    assert not proj[:, :, :-2].any()


# --------------------------------------------------------------------- two streams at once
@pytest.mark.parametrize("d", [32, 64])
def test_two_streams_at_the_same_time(d):
    """Training steps of both types in a graph on one stream, forwards, plain attention, a token over a
    cache and the rotary in a graph on another, replayed together several times: their intervals
    overlap and every output has the bits of the calls on their own."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    x, f = make(2, 6, 2, 1500, d, "bf16"), make(1, 4, 2, 500, d, "f32", 2)
    y = make(3, 4, 2, 2000, d, "bf16", 1)
    Q, K, V, lam, _ = y
    q, lens = Q[:, :, -1:].contiguous(), torch.tensor([2000, 0, 77], dtype=torch.int32, device="cuda")
    P, R, S = (torch.randn(2, 4, 1500, d, device="cuda").bfloat16() for _ in range(3))
    pos = torch.arange(2000, device="cuda", dtype=torch.int32)[None]
    freq, axis = torch.rand(d // 2, device="cuda"), torch.zeros(d // 2, dtype=torch.int32, device="cuda")

    def step(x):
        O, O2, lse = fbd.attn_diff_fwd(*x[:4])
        return (O, O2, lse, *fbd.attn_diff_bwd(*x[:4], O, O2, x[4], lse))

    def one():
        return (*step(x), *step(f))

    def other():
        return (fbd.attn_diff_decode(q, K, V, lam, lens), *step(y), *fbd.attn_fwd(P, R, S),
                *fbd.attn_rope((Q, K), pos, freq, axis))

    want = [one(), other()]
    torch.cuda.synchronize()
    times, graphs, got = 12, [], []
    for calls in (one, other):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            for _ in range(times):
                out = calls()
        graphs.append(gr)
        got.append(out)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for out in got:
            for t in out:
                t.zero_()
        start = torch.cuda.Event(enable_timing=True)
        ends = [[torch.cuda.Event(enable_timing=True) for _ in range(2)] for _ in range(2)]
        start.record()
        for st, gr, (a, b) in zip(streams, graphs, ends):
            st.wait_event(start)
            with torch.cuda.stream(st):
                a.record()
                gr.replay()
                b.record()
        torch.cuda.synchronize()
        (a0, a1), (b0, b1) = [[start.elapsed_time(e) for e in pair] for pair in ends]
        assert min(a1, b1) - max(a0, b0) > 0.5 * min(a1 - a0, b1 - b0), (a0, a1, b0, b1)
        for g, w in zip(got, want):
            for u, v in zip(g, w):
                assert torch.equal(u, v)
    fbd.attn_device_status()


# -------------------------------------------------------------- infinities among the keys
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64])
def test_an_infinite_score_is_its_own_maps(d, dtype):
    """Visible keys with an infinity in one map, their scores minus infinity: weight 0 in that map, the
    other map's as if nothing were there; over a cache and in the forward."""
    import diff_reference as R
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    B, H, g, N = 2, 4, 2, 200
    Q, K, V, lam, _ = make(B, H, g, N, d, dtype)
    Q[:, 0::2, :, 5], Q[:, 1::2, :, d - 1] = -Q[:, 0::2, :, 5].abs() - 0.5, Q[:, 1::2, :, d - 1].abs() + 0.5
    K[:, 0::2, 3::7, 5] = math.inf            # first maps
    K[:, 1::2, 4::9, d - 1] = -math.inf       # second maps
    lens = torch.tensor([N, 77], dtype=torch.int32, device="cuda")
    q = Q[:, :, -1:].contiguous()
    got = fbd.attn_diff_decode(q, K, V, lam, lens)
    want, tol = decode_reference(q, K, V, lam, lens, g)
    assert torch.isfinite(want).all() and torch.isfinite(got).all()
    assert ((got.double() - want).abs() <= tol).all()
    O, O2, lse = fbd.attn_diff_fwd(Q, K, V, lam)
    A, A2, L, P = R.forward(Q, K, V, lam, g, R.visible(N, "causal", device="cuda"))
    e, h = (2.0 ** -8 + R.FP32, 2.0 ** -8) if dtype == "bf16" else (R.FP32, 2.0 ** -24)
    mag = P @ V.double().unsqueeze(2).repeat_interleave(g, 1).abs()
    assert ((O2.double() - A2).abs() <= e * mag[:, :, 1] + h * A2.abs()).all()
    assert ((O.double() - A).abs() <= e * (mag[:, :, 0] + lam.abs()[:, None, None] * mag[:, :, 1]) + h * A.abs()).all()
    assert ((lse.double() - L).abs() <= R.FP32 * (1 + L.abs())).all()


# ------------------------------------------------------------------- far positions turned
def inverse_of_two_pi(bits=320):
    """1 / 2 pi as a fraction within 2^-bits, from Machin's formula pi = 16 arctan(1/5) - 4 arctan(1/239)."""
    one = 1 << (bits + 32)

    def arctan(n):
        term, total, k = one // n, 0, 0
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term, k = term // (n * n), k + 1
        return total

    return Fraction(one, 2 * (16 * arctan(5) - 4 * arctan(239)))


@pytest.mark.parametrize("paired", ["half", "neighbour"])
def test_angles_of_far_positions(paired):
    """Frequencies from 1e-30 to 2^40 of both signs at the farthest int32 positions, against angles
    reduced in rational arithmetic."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    d = 64
    freq = torch.tensor([1e-30, 1e-4, 0.03, 1.0, 6.9, 100.0, 1e4, 1e6, 2.0 ** 31, 2.0 ** 40, 3.3, 0.7, 12.5, 777.0, 4e8, 2.5],
                        dtype=torch.float32)
    freq = torch.cat([freq, -freq])
    pos = torch.tensor([0, 1, -1, 1000, -4097, 12000000, -99999999, (1 << 31) - 1, -(1 << 31)], dtype=torch.int32)
    N = pos.numel()
    x = torch.randn(1, 2, N, d, generator=torch.Generator().manual_seed(0))
    C = inverse_of_two_pi()
    angle = torch.empty(N, d // 2, dtype=torch.float64)
    for i, f in enumerate(freq.tolist()):
        for n, p in enumerate(pos.tolist()):
            turn = Fraction(f) * p * C
            angle[n, i] = 2 * math.pi * float(turn - round(turn))
    c, s = torch.cos(angle), torch.sin(angle)
    z = x.double()
    u, v = (z[..., :d // 2], z[..., d // 2:]) if paired == "half" else (z[..., 0::2], z[..., 1::2])
    a, b = u * c - v * s, u * s + v * c
    want = torch.cat([a, b], -1) if paired == "half" else torch.stack([a, b], -1).flatten(-2)
    got = fbd.attn_rope(x.cuda(), pos.cuda()[None], freq.cuda(), torch.zeros(d // 2, dtype=torch.int32, device="cuda"),
                        paired=paired).cpu().double()
    # the angle within 2^-32 of a turn (below 2^-29 radians) and its rounding to float32 (2^-24 of half a
    # turn, below 2^-22), of a pair's length below sqrt 2 of the largest coordinate; sine, cosine, two
    # products and their sum: each half a step, 2^-24, of terms no larger than that: 2^-21 in all
    tol = (2.0 ** -21 + math.sqrt(2) * (2.0 ** -29 + 2.0 ** -22)) * x.abs().max().item()
    assert (got - want).abs().max().item() <= tol


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
