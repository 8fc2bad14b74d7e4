"""Differential attention (forward, backward, one token over a cache) and the multi-axis
rotary on the GPU against plain 64-bit references; every output element within the bound
its roundings allow (tests/diff_reference.py)."""
import math

import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


def _t():
    import torch
    return torch


def dt(name):
    return {"bf16": _t().bfloat16, "f32": _t().float32}[name]


def make(B, H, g, N, d, dtype, seed=0, lam=None):
    torch = _t()
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt(dtype))  # noqa: E731
    Q, K, V, dO = r(B, 2 * H, N, d), r(B, 2 * H // g, N, d), r(B, H // g, N, 2 * d), r(B, H, N, 2 * d)
    if lam is None:
        lam = torch.linspace(-0.4, 1.1, H, device="cuda")
    return Q, K, V, lam, dO


def segments(B, N, mean, seed=1):
    torch = _t()
    gen = torch.Generator().manual_seed(seed)
    return (torch.rand(B, N, generator=gen) < 1.0 / mean).int().cumsum(1).int().cuda()


def check(got, want, what=""):
    """Every output within its bound; every element finite exactly where the reference is."""
    torch = _t()
    for name, x in got.items():
        ref, tol = want[name]
        err = (x.double() - ref).abs()
        assert torch.isfinite(x).all(), f"{what} {name} not finite"
        over = (err - tol).max().item() if x.numel() else 0.0
        assert over <= 0, f"{what} {name}: {over:.3e} past the bound, worst error {err.max().item():.3e}"
        n = ref.norm().item()
        if n == 0:
            assert err.max().item() == 0 or name == "lse", f"{what} {name}: zeros expected"


def run(x, **mask):
    import fwd_bwd_double_gb300 as fbd
    Q, K, V, lam, dO = x
    O, O2, lse = fbd.attn_diff_fwd(Q, K, V, lam, **mask)
    dQ, dK, dV, dlam = fbd.attn_diff_bwd(Q, K, V, lam, O, O2, dO, lse, **mask)
    fbd.attn_device_status()
    return dict(O=O, O2=O2, lse=lse, dQ=dQ, dK=dK, dV=dV, dlam=dlam)


def compare(B, H, g, N, d, dtype, mask="causal", window=0, mean=0, scale=0.0, seed=0, lam=None):
    import diff_reference as R
    import fwd_bwd_double_gb300 as fbd
    x = make(B, H, g, N, d, dtype, seed, lam)
    seg = segments(B, N, mean) if mean else None
    kw = dict(causal=mask != "full", window=window, scale=scale, bounds=fbd.attn_segment_bounds(seg) if mean else None)
    vis = R.visible(N, mask, window, seg, "cuda")
    check(run(x, **kw), R.with_bounds(*x, g, vis, scale or None), f"{(B, H, g, N, d, dtype, mask, window, mean)}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64])
@pytest.mark.parametrize("N", [1, 2, 17, 63, 64, 65, 127, 128, 129, 300])
def test_lengths(N, d, dtype):
    for mask in ("causal", "full"):
        compare(1, 2, 1, N, d, dtype, mask)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,g,N,d,mask,window,mean", [
    (2, 4, 2, 257, 64, "causal", 0, 0), (2, 3, 3, 200, 32, "full", 0, 0), (1, 4, 4, 700, 64, "causal", 0, 0),
    (1, 2, 1, 300, 64, "causal", 1, 0), (1, 2, 1, 300, 32, "causal", 2, 0), (2, 2, 2, 515, 64, "causal", 100, 0),
    (1, 2, 1, 900, 64, "causal", 129, 0), (1, 2, 1, 300, 64, "causal", 5000, 0),
    (2, 2, 1, 400, 64, "causal", 0, 1), (2, 2, 1, 600, 64, "causal", 0, 17), (3, 4, 2, 640, 32, "causal", 0, 90),
    (1, 6, 3, 1100, 64, "causal", 70, 300), (9, 3, 1, 140, 64, "causal", 0, 0), (1, 1, 1, 1500, 64, "full", 0, 0),
])
def test_masks_and_groups(B, H, g, N, d, mask, window, mean, dtype):
    compare(B, H, g, N, d, dtype, mask, window, mean)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scale_and_lambda_of_any_sign(dtype):
    torch = _t()
    compare(1, 3, 1, 200, 64, dtype, scale=0.05, lam=torch.tensor([0.0, -2.0, 3.0], device="cuda"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scores_far_apart(dtype):
    """Rows whose maximum moves late and by much: keys that grow along the sequence."""
    import diff_reference as R
    torch = _t()
    Q, K, V, lam, dO = make(1, 2, 1, 400, 64, dtype)
    ramp = torch.linspace(0.0, 3.0, 400, device="cuda")[:, None]
    x = (Q.abs(), (K.float().abs() * ramp).to(K.dtype), V, lam, dO)
    vis = R.visible(400, "causal", device="cuda")
    want = R.with_bounds(*x, 1, vis)
    got = run(x)
    # scores up to 3 * 64 * E|q||k| / 8 ~ 16 log2 e 2^5: the arguments' rounding is 2^5 / 2^6 of FP32's share
    check({k: got[k] for k in ("O", "O2", "lse", "dV")}, want)


def test_more_slices_than_a_grid_group():
    compare(3, 6, 2, 130, 64, "bf16")
    compare(3, 6, 2, 130, 64, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gradient_against_differences(dtype):
    """The directional derivative of sum(O dO) along the inputs, by central differences of the
    64-bit forward at the kernels' own (rounded) inputs."""
    import diff_reference as R
    torch = _t()
    x = make(1, 2, 2, 150, 32, dtype)
    got = run(x)
    Q, K, V, lam, dO = x
    vis = R.visible(150, "causal", device="cuda")
    bounds = R.with_bounds(*x, 2, vis)
    h = 1e-5
    for k, name in enumerate(("dQ", "dK", "dV", "dlam")):
        u = torch.randn(x[k].shape, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(k))
        f = []
        for sgn in (1, -1):
            y = [t.double() + sgn * h * u if i == k else t.double() for i, t in enumerate((Q, K, V, lam))]
            f.append((R.forward(*y, 2, vis)[0] * dO.double()).sum())
        slope = ((f[0] - f[1]) / (2 * h)).item()
        dot = (got[name].double() * u).sum().item()
        tol = (bounds[name][1] * u.abs()).sum().item() + 1e-7 * (1 + abs(f[0].item()))
        assert abs(slope - dot) <= tol, (name, slope, dot, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward_without_the_backwards_output(dtype):
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    Q, K, V, lam, _ = make(2, 2, 1, 200, 64, dtype)
    a = fbd.attn_diff_fwd(Q, K, V, lam)
    b = fbd.attn_diff_fwd(Q, K, V, lam, for_backward=False)
    assert b[1] is None and torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 100, 129])
def test_nothing_is_written_past_the_outputs(N, dtype):
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    B, H, g, d = 2, 2, 2, 64
    Q, K, V, lam, dO = make(B, H, g, N, d, dtype)

    def guarded(shape, dtype):
        n = math.prod(shape)
        buf = torch.full((n + 256,), 7.0, dtype=dtype, device="cuda")
        return buf, buf[128:128 + n].view(shape)

    bufs = {}
    for name, shape, t in (("O", dO.shape, Q.dtype), ("O2", dO.shape, Q.dtype), ("lse", Q.shape[:3], torch.float32),
                           ("dQ", Q.shape, Q.dtype), ("dK", K.shape, Q.dtype), ("dV", V.shape, Q.dtype),
                           ("dlam", lam.shape, torch.float32)):
        bufs[name] = guarded(tuple(shape), t)
    v = {k: b[1] for k, b in bufs.items()}
    fbd.attn_diff_fwd(Q, K, V, lam, O=v["O"], O2=v["O2"], lse=v["lse"])
    desc = fbd.AttnDesc(B, H, N, d, 0.0, 1, fbd.ATTN_BF16 if dtype == "bf16" else fbd.ATTN_F32, g, 0, None, None)
    need = fbd.attn_diff_bwd_workspace_bytes(desc)
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")  # float NaNs
    fbd.attn_diff_bwd(Q, K, V, lam, v["O"], v["O2"], dO, v["lse"], dQ=v["dQ"], dK=v["dK"], dV=v["dV"], dlam=v["dlam"],
                      workspace=ws[:need])
    torch.cuda.synchronize()
    for name, (buf, view) in bufs.items():
        assert (buf[:128] == 7).all() and (buf[128 + view.numel():] == 7).all(), name
    assert (ws[need:] == 0xFF).all()
    want = run((Q, K, V, lam, dO))
    for name in bufs:
        assert torch.equal(v[name], want[name]), name


def test_repeats_bit_for_bit():
    """Every output is the same on every call."""
    torch = _t()
    for dtype in ("bf16", "f32"):
        x = make(2, 4, 2, 700, 64, dtype)
        a, b = run(x), run(x)
        for name in a:
            assert torch.equal(a[name], b[name]), (dtype, name)


def test_smallest_scales():
    """A scale whose product with every score vanishes: uniform weights over the visible keys."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    Q, K, V, lam, _ = make(1, 2, 1, 300, 64, "bf16")
    O, O2, lse = fbd.attn_diff_fwd(Q, K, V, lam, scale=1.2e-38)
    n = torch.arange(1, 301, device="cuda", dtype=torch.float64)
    want = V.double().cumsum(2) / n[:, None]
    # P = 1 exactly; O2 = the sum of bf16 values in fp32, 1 / l and their product, then one bf16 rounding
    size = V.double().abs().cumsum(2) / n[:, None]
    assert ((O2.double() - want).abs() <= 2**-8 * want.abs() + 300 * 2**-24 * size).all()
    assert ((lse.double() - n.log()).abs() <= 2**-22 * (1 + n.log())).all()
    assert torch.isfinite(O).all()


def test_given_streams(monkeypatch):
    """The stream a call runs on: an object, its handle, the default stream's handle 0 under another
    stream, keywords in any order."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    Q, K, V, lam, _ = make(1, 2, 1, 130, 64, "bf16")
    seen = []
    launch = fbd._launch
    monkeypatch.setattr(fbd, "_launch", lambda *a: (seen.append(torch.cuda.current_stream()), launch(*a)))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        fbd.attn_diff_fwd(Q, K, V, lam)
        fbd.attn_diff_fwd(Q, K, V, lam, stream=0)
    fbd.attn_diff_fwd(scale=0.5, Q=Q, K=K, V=V, lam=lam, stream=st)
    fbd.attn_diff_fwd(Q, K, V, lam, stream=st.cuda_stream)
    assert [s.cuda_stream for s in seen] == [st.cuda_stream, 0, st.cuda_stream, st.cuda_stream]
    torch.cuda.synchronize()


@pytest.mark.parametrize("d", [32, 64])
def test_calls_at_once(d):
    """Training steps on one stream, forwards of plain attention and a token over a cache on another:
    the bits of the calls on their own."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    x = make(2, 6, 2, 1500, d, "bf16")
    Q, K, V, lam, _ = make(3, 4, 2, 2000, d, "bf16", 1)
    q, lens = Q[:, :, -1:].contiguous(), torch.tensor([2000, 0, 77], dtype=torch.int32, device="cuda")
    P, R, S = (torch.randn(2, 4, 1500, d, device="cuda").bfloat16() for _ in range(3))

    def other():
        return (fbd.attn_diff_decode(q, K, V, lam, lens), *fbd.attn_diff_fwd(Q, K, V, lam), *fbd.attn_fwd(P, R, S))

    want, want_other = run(x), other()
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    got, got_other = [], []
    for _ in range(4):
        with torch.cuda.stream(a):
            got.append(run(x))
        with torch.cuda.stream(b):
            got_other.append(other())
    torch.cuda.synchronize()
    fbd.attn_device_status()
    for g, o in zip(got, got_other):
        for k in want:
            assert torch.equal(g[k], want[k]), k
        for u, v in zip(o, want_other):
            assert torch.equal(u, v)


def test_streams_graphs_and_views_of_lam():
    """On another stream; captured twice over one workspace and replayed in turn on new data; lam a
    slice of a larger tensor (4-byte aligned)."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    x = make(1, 3, 1, 300, 64, "bf16")
    big = torch.cat([x[3].new_zeros(1), x[3]])
    x = (*x[:3], big[1:], x[4])
    want = run(x)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = run(x)
    for k in got:
        assert torch.equal(got[k], want[k]), k
    for given in (st, st.cuda_stream):  # the stream as an argument, an object or its handle
        O, O2, lse = fbd.attn_diff_fwd(*x[:4], stream=given)
        dQ, dK, dV, dlam = fbd.attn_diff_bwd(*x[:4], O, O2, x[4], lse, stream=given)
        st.synchronize()
        for k, v in dict(O=O, O2=O2, lse=lse, dQ=dQ, dK=dK, dV=dV, dlam=dlam).items():
            assert torch.equal(v, want[k]), k
    desc = fbd.AttnDesc(1, 3, 300, 64, 0.0, 1, fbd.ATTN_BF16, 1, 0, None, None)
    ws = torch.empty(fbd.attn_diff_bwd_workspace_bytes(desc), dtype=torch.uint8, device="cuda")

    def step(x):
        O, O2, lse = fbd.attn_diff_fwd(*x[:4])
        return (O, *fbd.attn_diff_bwd(*x[:4], O, O2, x[4], lse, workspace=ws))

    graphs = []
    for seed in (1, 2):
        y = tuple(t.clone() for t in make(1, 3, 1, 300, 64, "bf16", seed))
        step(y)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            out = step(y)
        graphs.append((gr, y, out))
    for seed in (3, 4, 5):
        for k, (gr, y, out) in enumerate(graphs):
            new = make(1, 3, 1, 300, 64, "bf16", seed + 10 * k)
            for a, b in zip(y, new):
                a.copy_(b)
            gr.replay()
            w = run(new)
            torch.cuda.synchronize()
            for a, name in zip(out, ("O", "dQ", "dK", "dV", "dlam")):
                assert torch.equal(a, w[name]), name


def test_empty_gradient_of_lambda_is_zero():
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    Q, K, V, lam, dO = (t[:, :, :0].contiguous() if t.dim() == 4 else t for t in make(2, 3, 1, 4, 32, "bf16"))
    O, O2, lse = fbd.attn_diff_fwd(Q, K, V, lam)
    dlam = torch.full_like(lam, 5.0)
    dQ, dK, dV, dlam = fbd.attn_diff_bwd(Q, K, V, lam, O, O2, dO, lse, dlam=dlam)
    assert dQ.numel() == 0 and (dlam == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_2_31_elements(dtype):
    """16 heads of a 2^20-token window: Q and V alone have 2^31 elements.  The last head is what it is
    alone, bit for bit."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    N, d, W = 1 << 20, 64, 40
    H = 16 if dtype == "bf16" else 17
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GB of device memory")
    gen = torch.Generator(device="cuda").manual_seed(0)

    def big(heads, width):  # the last head's values random, the others' zero
        x = torch.zeros(1, heads, N, width, dtype=dt(dtype), device="cuda")
        x[:, -(heads // H):] = torch.randn(1, heads // H, N, width, generator=gen, device="cuda").to(dt(dtype))
        return x

    Q, K, V, dO = big(2 * H, d), big(2 * H, d), big(H, 2 * d), big(H, 2 * d)
    lam = torch.full((H,), 0.5, device="cuda")
    a = run((Q, K, V, lam, dO), window=W)
    last = tuple(t[:, -(t.shape[1] // H):].contiguous() for t in (Q, K, V)) + (lam[-1:], dO[:, -1:].contiguous())
    b = run(last, window=W)
    for k in b:
        got = a[k][-1:] if k == "dlam" else a[k][:, -(a[k].shape[1] // H):]
        assert torch.equal(got, b[k]), k
    if dtype == "bf16":  # and over a cache of that size
        lens = torch.tensor([N], dtype=torch.int32, device="cuda")
        o = fbd.attn_diff_decode(Q[:, :, -1:].contiguous(), K, V, lam, lens)
        want, tol = decode_reference(last[0][:, :, -1:], last[1], last[2], last[3], lens, 1)
        assert ((o[:, -1:].double() - want).abs() <= tol).all()
        pos = torch.arange(N, device="cuda", dtype=torch.int32)[None]
        freq, axis = torch.rand(d // 2, device="cuda"), torch.zeros(d // 2, dtype=torch.int32, device="cuda")
        r = fbd.attn_rope(Q, pos, freq, axis)
        assert torch.equal(r[:, -2:], fbd.attn_rope(last[0], pos, freq, axis))


# ------------------------------------------------------------------ one token over a cache
def decode_reference(Q, K, V, lam, lens, g, window=0):
    torch = _t()
    B, H2, _, d = Q.shape
    H, cap = H2 // 2, K.shape[2]
    out, tol = torch.zeros(2, B, H, 1, 2 * d, dtype=torch.float64, device="cuda")
    bf16 = Q.dtype == torch.bfloat16
    e, h = ((2.0 ** -8 + 1e-5), 2.0 ** -8) if bf16 else (1e-5, 2.0 ** -24)
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        lo = max(0, n - window) if window else 0
        if n == 0:
            continue
        for hh in range(H):
            v = V[b, hh // g, lo:n].double()
            o = []
            mag = 0.0
            for m in range(2):
                p = torch.softmax(K[b, 2 * (hh // g) + m, lo:n].double() @ Q[b, 2 * hh + m, 0].double() / math.sqrt(d), 0)
                o.append(p @ v)
                mag = mag + (1.0 if m == 0 else abs(lam[hh].item())) * (p @ v.abs())
            out[b, hh, 0] = o[0] - lam[hh].double() * o[1]
            tol[b, hh, 0] = e * mag + h * out[b, hh, 0].abs()
    return out, tol


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,g,cap,d,window", [
    (1, 1, 1, 1, 64, 0), (2, 2, 1, 40, 32, 0), (3, 4, 2, 65, 64, 0), (2, 8, 8, 1000, 64, 0), (2, 9, 9, 300, 32, 0),
    (1, 20, 20, 513, 64, 0), (1, 6, 1, 5000, 64, 0), (5, 4, 4, 2049, 64, 100), (4, 2, 1, 700, 32, 1), (2, 3, 1, 90, 64, 4000),
    (1, 33, 33, 130, 64, 0), (40, 4, 2, 600, 64, 0), (1, 1, 1, 40000, 32, 0),
])
def test_decode(B, H, g, cap, d, window, dtype):
    """Ragged lengths, among them none, one, a whole cache and bounds outside it; the cache rows no
    token sees hold NaN and infinities."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    gen = torch.Generator(device="cuda").manual_seed(B * cap)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt(dtype))  # noqa: E731
    Q, K, V = r(B, 2 * H, 1, d), r(B, 2 * H // g, cap, d), r(B, H // g, cap, 2 * d)
    lam = torch.linspace(-0.3, 0.9, H, device="cuda")
    lens = torch.randint(1, cap + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
    special = [cap, 0, 1, cap + 7, -3]
    for b in range(1, min(B, 6)):
        lens[b] = special[b - 1]
    for b in range(B):
        n = min(max(int(lens[b]), 0), cap)
        lo = max(0, n - window) if window else 0
        K[b, :, n:], V[b, :, n:] = math.nan, math.inf
        K[b, :, :lo], V[b, :, :lo] = math.inf, math.nan
    got = fbd.attn_diff_decode(Q, K, V, lam, lens, window=window)
    fbd.attn_device_status()
    want, tol = decode_reference(Q, K, V, lam, lens, g, window)
    assert torch.isfinite(got).all()
    assert ((got.double() - want).abs() <= tol).all(), (got.double() - want).abs().max()
    assert torch.equal(got, fbd.attn_diff_decode(Q, K, V, lam, lens, window=window))


def test_decode_is_the_last_row_of_the_forward():
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    for N in (1, 31, 200):
        Q, K, V, lam, _ = make(2, 4, 2, N, 64, "f32")
        O, _, _ = fbd.attn_diff_fwd(Q, K, V, lam)
        lens = torch.full((2,), N, dtype=torch.int32, device="cuda")
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        o = fbd.attn_diff_decode(Q[:, :, -1:].contiguous(), K, V, lam, lens, stream=st)
        st.synchronize()
        assert (o - O[:, :, -1:]).abs().max() <= 1e-5 * V.abs().max() * 2.1


def test_decode_without_a_cache_gives_zeros():
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    Q, K, V, lam, _ = make(2, 3, 1, 1, 64, "bf16")
    O = torch.full((2, 3, 1, 128), 9.0, dtype=Q.dtype, device="cuda")
    fbd.attn_diff_decode(Q, K[:, :, :0].contiguous(), V[:, :, :0].contiguous(), lam,
                         torch.zeros(2, dtype=torch.int32, device="cuda"), O=O)
    assert (O == 0).all()


def test_decode_in_a_graph_follows_the_lengths():
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    Q, K, V, lam, _ = make(3, 4, 2, 1, 64, "bf16")
    _, K, V, _, _ = make(3, 4, 2, 3000, 64, "bf16", seed=1)
    lens = torch.tensor([5, 0, 900], dtype=torch.int32, device="cuda")
    fbd.attn_diff_decode(Q, K, V, lam, lens)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        out = fbd.attn_diff_decode(Q, K, V, lam, lens)
    for step in ([6, 1, 901], [3000, 64, 0], [1, 33, 2999]):
        lens.copy_(torch.tensor(step, dtype=torch.int32))
        gr.replay()
        assert torch.equal(out, fbd.attn_diff_decode(Q, K, V, lam, lens))


# ------------------------------------------------------------------------------- rotary
def rope_bound(x, want, inverse=False):
    """Half a step of the output, and three fp32 roundings of terms no larger than the pair."""
    torch = _t()
    h = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    return h * want.abs() + 2.0 ** -21 * x.double().abs().max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("paired", ["half", "neighbour"])
@pytest.mark.parametrize("B,heads,N,d,axes", [(1, 1, 1, 32, 1), (2, 3, 17, 64, 3), (3, 2, 300, 96, 2), (1, 5, 129, 128, 4),
                                              (2, 1, 33, 256, 2)])
def test_rope(B, heads, N, d, axes, paired, dtype):
    import diff_reference as R
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    gen = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(B, heads, N, d, generator=gen, device="cuda").to(dt(dtype))
    pos = torch.randint(1 - (1 << 31), (1 << 31) - 1, (axes, B, N), generator=gen, device="cuda").int()
    pos[:, :, ::2] %= 1000
    freq = torch.rand(d // 2, generator=gen, device="cuda") * 7 - 1
    freq[::3] = 10000.0 ** -torch.rand(freq[::3].shape, generator=gen, device="cuda")
    axis = torch.randint(-1, axes + 1, (d // 2,), generator=gen, device="cuda").int()  # out of range: copied
    for inverse in (False, True):
        want = R.rope(x, pos, freq, axis, paired, inverse)
        got = fbd.attn_rope(x, pos, freq, axis, paired=paired, inverse=inverse)
        # the fraction of a turn per step is rounded twice (1.5 2^-53), the reference's angle once: times 2^31 steps
        # and sqrt 2 for the pair, below 2^-17 of a radian
        slack = x.double().abs().max() * 2.0 ** -17
        assert ((got.double() - want).abs() <= rope_bound(x, want) + slack).all()
        near = (pos.abs() < 1000).all(0)[:, None, :, None].expand_as(x)
        assert ((got.double() - want).abs() <= rope_bound(x, want))[near].all()
    copied = (axis < 0) | (axis >= axes)
    cols = torch.cat([copied, copied]) if paired == "half" else copied.repeat_interleave(2)
    assert torch.equal(got[..., cols], x[..., cols])


def test_rope_views_in_place_and_shared_positions():
    """Queries and keys as views of one projection's [B, N, heads, d] output, written contiguous, back
    into the buffer's own layout, and in place; positions shared by the batch."""
    import diff_reference as R
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    B, N, d, hq, hk = 2, 77, 64, 6, 2
    qkv = torch.randn(B, N, hq + 2 * hk, d, device="cuda").bfloat16()
    keep = qkv.clone()
    q, k = qkv[:, :, :hq].transpose(1, 2), qkv[:, :, hq:hq + hk].transpose(1, 2)
    pos = torch.randint(0, 500, (2, N), device="cuda").int()
    freq = 100.0 ** -torch.linspace(0, 1, d // 2, device="cuda")
    axis = (torch.arange(d // 2, device="cuda") % 2).int()
    wq, wk = (R.rope(t, pos[:, None].expand(2, B, N), freq, axis) for t in (q, k))
    a, b = fbd.attn_rope((q, k), pos, freq, axis)
    assert a.is_contiguous() and b.is_contiguous() and torch.equal(qkv, keep)
    assert ((a.double() - wq).abs() <= rope_bound(q, wq)).all() and ((b.double() - wk).abs() <= rope_bound(k, wk)).all()
    # the same with positions of every batch row written out
    c = fbd.attn_rope(q, pos[:, None].expand(2, B, N).contiguous(), freq, axis)
    assert torch.equal(a, c)
    # into views of another [B, N, heads, d] buffer
    out = torch.full_like(qkv, 3.0)
    fbd.attn_rope((q, k), pos, freq, axis, outs=(out[:, :, :hq].transpose(1, 2), out[:, :, hq:hq + hk].transpose(1, 2)))
    assert torch.equal(out[:, :, :hq].transpose(1, 2), a) and torch.equal(out[:, :, hq:hq + hk].transpose(1, 2), b)
    assert (out[:, :, hq + hk:] == 3).all()
    # a broadcast input
    e = fbd.attn_rope(q[:, :1].expand(B, 3, N, d), pos, freq, axis)
    assert all(torch.equal(e[:, u], a[:, 0]) for u in range(3))
    # in place
    fbd.attn_rope((q, k), pos, freq, axis, outs=(q, k))
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(qkv[:, :, hq + hk:], keep[:, :, hq + hk:])


def test_rope_feeds_plain_attention_and_its_second_backward():
    """The turn is linear and orthogonal: the gradients of the turned queries go back through the
    inverse turn (attn_bwd), checked against autograd in 64 bits."""
    import diff_reference as R
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    B, H, N, d = 1, 2, 150, 64
    gen = torch.Generator(device="cuda").manual_seed(0)
    Q, K, V, dO = (torch.randn(B, H, N, d, generator=gen, device="cuda") for _ in range(4))
    pos = torch.stack([torch.arange(N), torch.arange(N) // 10]).int().cuda()
    freq = 50.0 ** -torch.linspace(0, 1, d // 2, device="cuda")
    axis = (torch.arange(d // 2) // 16).int().cuda()
    q, k = fbd.attn_rope((Q, K), pos, freq, axis)
    O, lse = fbd.attn_fwd(q, k, V)
    dq, dk, dV = fbd.attn_bwd(q, k, V, O, dO, lse)
    dQ, dK = fbd.attn_rope((dq, dk), pos, freq, axis, inverse=True)
    x = [t.double().requires_grad_() for t in (Q, K, V)]
    p3 = pos[:, None].expand(2, B, N)
    S = R.rope(x[0], p3, freq, axis) @ R.rope(x[1], p3, freq, axis).transpose(-1, -2) / math.sqrt(d)
    S = S.masked_fill(~R.visible(N, "causal", device="cuda")[:, None], -math.inf)
    want = torch.autograd.grad((torch.softmax(S, -1) @ x[2] * dO.double()).sum(), x)
    for got, w in zip((dQ, dK, dV), want):
        assert (got.double() - w).norm() <= 1e-5 * w.norm()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_layer_from_projection_to_gradients_and_one_more_token(dtype):
    """The operators together: projection -> rotary (time, height, width) -> differential attention ->
    backward -> rotary back, against autograd in 64 bits; then the next token over the cache."""
    import diff_reference as R
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    B, H, g, N, d = 2, 4, 2, 193, 64
    Hkv = H // g
    gen = torch.Generator(device="cuda").manual_seed(0)
    proj = torch.randn(B, N + 1, 2 * H + 2 * Hkv, d, generator=gen, device="cuda").to(dt(dtype))
    V = torch.randn(B, Hkv, N + 1, 2 * d, generator=gen, device="cuda").to(dt(dtype))
    dO = torch.randn(B, H, N, 2 * d, generator=gen, device="cuda").to(dt(dtype))
    lam = torch.tensor([0.8, 0.2, 0.5, -0.1], device="cuda")
    n = torch.arange(N + 1, device="cuda")
    pos = torch.stack([n // 16, n // 4 % 4, n % 4]).int()
    freq = 100.0 ** -torch.linspace(0, 1, d // 2, device="cuda")
    axis = (torch.arange(d // 2, device="cuda") * 3 // (d // 2)).int()
    q_all, k_all = proj[:, :, :2 * H].transpose(1, 2), proj[:, :, 2 * H:].transpose(1, 2)
    # training on the first N tokens
    p = pos[:, :N].contiguous()
    v = V[:, :, :N].contiguous()
    q, k = fbd.attn_rope((q_all[:, :, :N], k_all[:, :, :N]), p, freq, axis)
    O, O2, lse = fbd.attn_diff_fwd(q, k, v, lam)
    dq, dk, dV, dlam = fbd.attn_diff_bwd(q, k, v, lam, O, O2, dO, lse)
    grad = torch.zeros_like(proj)
    fbd.attn_rope((dq, dk), p, freq, axis, inverse=True,
                  outs=(grad[:, :N, :2 * H].transpose(1, 2), grad[:, :N, 2 * H:].transpose(1, 2)))
    x = [proj[:, :N].double().requires_grad_(), v.double().requires_grad_(), lam.double().requires_grad_()]
    p3 = p[:, None].expand(3, B, N)
    vis = R.visible(N, "causal", device="cuda")
    want_O, _, _, _ = R.forward(R.rope(x[0][:, :, :2 * H].transpose(1, 2), p3, freq, axis),
                                R.rope(x[0][:, :, 2 * H:].transpose(1, 2), p3, freq, axis), x[1], x[2], g, vis)
    want = torch.autograd.grad((want_O * dO.double()).sum(), x)
    # roundings of the turned q and k move every score by 2^-8 |q||k| / 8 at most (each 2^-8 of a term of
    # |q.k| / 8 ~ N(0, 1), 64 independent terms: about 2^-8), so P by that much relatively: with P's, dS's,
    # O's and the gradients' own roundings eight half steps of 2^-8 in all
    tol = 8 * 2.0 ** -8 if dtype == "bf16" else 2e-5
    for got, w in ((O, want_O), (grad[:, :N], want[0]), (dV, want[1]), (dlam, want[2])):
        assert (got.double() - w).norm() <= tol * w.norm()
    # one more token: its key and value into the cache, then its row
    K = torch.full((B, 2 * Hkv, 256, d), math.nan, device="cuda", dtype=proj.dtype)
    Vc = torch.full((B, Hkv, 256, 2 * d), math.nan, device="cuda", dtype=proj.dtype)
    K[:, :, :N], Vc[:, :, :N + 1] = k, V
    last = pos[:, N:].contiguous()
    q1, _ = fbd.attn_rope((q_all[:, :, N:], k_all[:, :, N:]), last, freq, axis,
                          outs=(torch.empty(B, 2 * H, 1, d, device="cuda", dtype=proj.dtype), K[:, :, N:N + 1]))
    o = fbd.attn_diff_decode(q1, K, Vc, lam, torch.full((B,), N + 1, dtype=torch.int32, device="cuda"))
    p3 = pos[:, None].expand(3, B, N + 1)
    full, _, _, _ = R.forward(R.rope(q_all, p3, freq, axis), R.rope(k_all, p3, freq, axis), V, lam, g,
                              R.visible(N + 1, "causal", device="cuda"))
    assert (o.double() - full[:, :, N:]).norm() <= tol * full[:, :, N:].norm()
