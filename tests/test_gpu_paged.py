"""Normed heads, appends to a paged cache and the attention over it on the GPU against plain 64-bit
references; every output element within the bound its roundings allow (tests/paged_reference.py)."""
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


def within(got, want, what=""):
    """got within its bound of want = (value, bound), finite wherever the value is, equal where it is infinite."""
    torch = _t()
    ref, tol = want
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isfinite(got), fin), f"{what}: finite elsewhere"
    assert torch.equal(got[~fin].double(), ref[~fin].double()), what
    err = (got.double() - ref).abs()[fin]
    over = (err - tol[fin]).max().item() if err.numel() else 0.0
    assert over <= 0, f"{what}: {over:.3e} past the bound, worst error {err.max().item():.3e}"


def randn(*shape, dtype, seed=0):
    torch = _t()
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(dtype)


def tables(B, N, d, axes, far=False, shared=False):
    torch = _t()
    gen = torch.Generator(device="cuda").manual_seed(9)
    top = (1 << 31) - 1 if far else 3000
    pos = torch.randint(-5 if not far else -top, top, (axes, N) if shared else (axes, B, N), generator=gen, device="cuda",
                        dtype=torch.int64).int()
    freq = (10000.0 ** (-torch.arange(d // 2, device="cuda", dtype=torch.float64) / (d // 2))).float()
    axis = (torch.arange(d // 2, device="cuda") % (axes + 1) - 1).int()  # some pairs (-1) are not turned
    return pos, freq, axis


# ------------------------------------------------------------------------------ normed heads
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("B,N,HQ,HK,axes,paired", [(1, 1, 1, 1, 1, "half"), (2, 37, 5, 2, 3, "neighbour"),
                                                    (3, 130, 9, 3, 2, "half"), (1, 700, 12, 1, 1, "neighbour")])
def test_norm_and_its_gradient(B, N, HQ, HK, axes, paired, d, dtype):
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    qk = 2 * randn(B, N, HQ + HK, d, dtype=dt(dtype))
    xs = [t.transpose(1, 2) for t in qk.split([HQ, HK], 2)]
    ws = [1 + 0.3 * randn(d, dtype=torch.float32, seed=k) for k in (1, 2)]
    pos, freq, axis = tables(B, N, d, axes)
    cs = R.cos_sin(pos, freq, axis)
    ys = fbd.attn_qk_norm(xs, ws, pos, freq, axis, paired=paired)
    dys = [randn(*x.shape, dtype=dt(dtype), seed=3 + k) for k, x in enumerate(xs)]
    dxs, dws = fbd.attn_qk_norm_bwd(xs, dys, ws, pos, freq, axis, paired=paired)
    fbd.attn_device_status()
    for k, (x, w) in enumerate(zip(xs, ws)):
        within(ys[k], R.norm(x, w, cs, paired), f"y[{k}]")
        dx, dw = R.norm_bwd(x, w, dys[k], cs, paired)
        within(dxs[k], dx, f"dx[{k}]")
        within(dws[k], dw, f"dw[{k}]")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_without_weights_or_turn_shared_positions_and_eps(dtype):
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    x, dy = randn(2, 3, 50, 64, dtype=dt(dtype)), randn(2, 3, 50, 64, dtype=dt(dtype), seed=1)
    within(fbd.attn_qk_norm(x), R.norm(x, None, None), "plain")
    dx, dw = fbd.attn_qk_norm_bwd(x, dy)
    assert dw is None
    within(dx, R.norm_bwd(x, None, dy, None)[0], "dx")
    pos, freq, axis = tables(2, 50, 64, 2, shared=True)
    cs = R.cos_sin(pos[:, None].expand(-1, 2, -1), freq, axis)
    w = randn(64, dtype=torch.float32, seed=2)
    within(fbd.attn_qk_norm(x, w, pos, freq, axis, eps=0.5), R.norm(x, w, cs, eps=0.5), "eps")
    dx, dw = fbd.attn_qk_norm_bwd(x, dy, w, pos, freq, axis, eps=0.5)
    want = R.norm_bwd(x, w, dy, cs, eps=0.5)
    within(dx, want[0], "dx eps")
    within(dw, want[1], "dw eps")
    # a head of zeros: zeros, and dx = eps^-1/2 w dz
    z = torch.zeros_like(x)
    assert not fbd.attn_qk_norm(z, w).any()
    within(fbd.attn_qk_norm_bwd(z, dy, w)[0], R.norm_bwd(z, w, dy, None)[0], "dx at zero")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_views_in_place_and_tensors_without_heads(dtype):
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    B, N, d = 2, 77, 96
    w = 1 + 0.1 * randn(d, dtype=torch.float32)
    qkv = randn(B, N, 7, d, dtype=dt(dtype))
    keep = qkv.clone()
    q, k = qkv[:, :, :4].transpose(1, 2), qkv[:, :, 4:6].transpose(1, 2)
    none = qkv[:, :, :0].transpose(1, 2)
    out = fbd.attn_qk_norm((q, none, k), (w, w, w), outs=(q, none, k))   # in place; V's head is left alone
    assert out[0] is q
    for got, x in ((q, keep[:, :, :4]), (k, keep[:, :, 4:6])):
        within(got, R.norm(x.transpose(1, 2), w, None), "in place")
    assert torch.equal(qkv[:, :, 6], keep[:, :, 6])
    x = keep[:, :, :4].transpose(1, 2)
    dy = randn(B, N, 4, d, dtype=dt(dtype), seed=4).transpose(1, 2)
    want = R.norm_bwd(x, w, dy, None)
    over_dy, over_x = dy.clone(), x.clone()
    for given, kw in ((x, dict(dys=over_dy, dxs=over_dy)), (over_x, dict(dys=dy, dxs=over_x))):
        dx, dw = fbd.attn_qk_norm_bwd(given, weights=w, **kw)
        within(dx, want[0], "dx in place")
        within(dw, want[1], "dw")
    (_, dxn), (_, dwn) = fbd.attn_qk_norm_bwd((x, none), (dy, none), (w, w))
    assert dxn.numel() == 0 and not dwn.any()
    empty = qkv[:, :0].transpose(1, 2)
    dx, dw = fbd.attn_qk_norm_bwd(empty, empty, w)
    assert dx.numel() == 0 and not dw.any()


def test_norm_gradient_against_differences():
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    x, dy = randn(1, 2, 40, 64, dtype=torch.float32), randn(1, 2, 40, 64, dtype=torch.float32, seed=1)
    w = 1 + 0.2 * randn(64, dtype=torch.float32, seed=2)
    pos, freq, axis = tables(1, 40, 64, 2)
    cs = R.cos_sin(pos, freq, axis)
    dx, dw = fbd.attn_qk_norm_bwd(x, dy, w, pos, freq, axis)
    h = 1e-5
    for k, (t, grad) in enumerate(((x, dx), (w, dw))):
        u = torch.randn(t.shape, dtype=torch.float64, device="cuda", generator=torch.Generator("cuda").manual_seed(k))
        f = []
        for sgn in (1, -1):
            xx, ww = (a.double() + sgn * h * u if a is t else a.double() for a in (x, w))
            z = xx * (xx.square().mean(-1, keepdim=True) + 1e-6) ** -0.5 * ww
            f.append((R.turn(z, cs, "half")[0] * dy.double()).sum().item())
        # the differences' own error: h^2 times a third derivative of order 10 |terms|, and the gradient's 1e-5
        mag = (grad.double().abs() * u.abs()).sum().item()
        assert abs((f[0] - f[1]) / (2 * h) - (grad.double() * u).sum().item()) <= 2e-5 * mag


# ---------------------------------------------------------------------------------- appends
def append_case(new, lens, page, heads, d, dtype, packed=True, normed=True, turned=True, with_q=True, axes=0, **kw):
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    x = R.Batch(new, lens, page, heads, d, dt(dtype), packed=packed, **kw)
    B, N = x.rows
    k, v = (x.randn(B, N, x.Hkv, d).transpose(1, 2) for _ in range(2))
    ws = [1 + 0.2 * randn(d, dtype=torch.float32, seed=k) for k in (5, 6)] if normed else None
    own = torch.zeros(1, B, N, dtype=torch.int32, device="cuda")
    for b in range(len(new)):
        r, rows = x.place(b)
        own[0, r, rows] = max(lens[b], 0) - new[b] + torch.arange(new[b], device="cuda", dtype=torch.int32)
    pos = freq = axis = cs = None
    if turned:
        pos, freq, axis = tables(B, N, d, max(axes, 1))
        cs = R.cos_sin(pos if axes else own, freq, axis)
        pos = pos if axes else None
    K0, V0, Q0 = x.K.clone(), x.V.clone(), x.Q.clone()
    out = torch.full_like(x.Q, 7.0) if with_q else None
    got = fbd.attn_cache_append(k, v, x.cache, x.lens, x.cu, Q=x.Q if with_q else None, Q_out=out, weights=ws, pos=pos, freq=freq,
                                axis=axis)
    fbd.attn_device_status()
    assert got is out

    def made(t, w):
        if normed:
            return R.norm(t, w, cs)
        y, mag = R.turn(t.double(), cs, "half")
        return y, (R.NORM * mag if turned else 0 * mag) + (R.half_step(t.dtype) * y.abs() if turned else 0)

    kw_, kt = made(k, ws[1] if normed else None)
    hit = torch.zeros(x.K.shape[0], page, dtype=torch.bool, device="cuda")
    for b in range(len(new)):
        r, rows = x.place(b)
        for t in range(new[b]):
            p = max(lens[b], 0) - new[b] + t
            if p < 0 or p // page >= x.width:
                continue
            pg = int(x.table[b, p // page])
            if not 0 <= pg < x.K.shape[0]:
                continue
            hit[pg, p % page] = True
            i = rows.start + t
            within(x.K[pg, :, p % page], (kw_[r, :, i], kt[r, :, i]), f"key {b} {t}")
            assert torch.equal(x.V[pg, :, p % page], v[r, :, i])
    away = ~hit[:, None, :, None].expand(x.K.shape)
    assert torch.equal(x.K[away], K0[away]) and torch.equal(x.V[away], V0[away])  # nothing else is written
    if with_q:
        qw, qt = made(Q0, ws[0] if normed else None)
        inside = torch.zeros(B, N, dtype=torch.bool, device="cuda")
        for b in range(len(new)):
            inside[x.place(b)] = True
        m = inside[:, None, :, None].expand(out.shape)
        within(out[m], (qw[m], qt[m]), "Q_out")
        assert (out[~m] == 7.0).all()  # rows of no sequence


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 256])
def test_append_ragged(d, dtype):
    append_case([5, 0, 1, 33, 16], [40, 9, 1, 33, 100], 16, (6, 2), d, dtype, behind=3)
    append_case([7, 50], [7, 113], 48, (4, 4), d, dtype, token_major=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(normed=False), dict(turned=False), dict(normed=False, turned=False), dict(with_q=False),
                                dict(axes=3), dict(packed=False), dict(packed=False, axes=2), dict(token_major=True)])
def test_append_forms(kw, dtype):
    append_case([4, 4, 4], [20, 4, 77], 32, (4, 2), 64, dtype, **kw)


def test_append_outside_the_table_or_the_cache():
    """Tokens before the first key, behind the table's last page or on no page are left out; their queries are not."""
    append_case([8, 40], [3, 60], 16, (2, 1), 64, "bf16", width=2)
    append_case([8, 40], [-4, 60], 16, (2, 1), 64, "bf16", width=2)


# -------------------------------------------------------------------------------- attention
def attend(x, causal=True, window=0, scale=0.0, max_new=None, check=True, sums=False, **kw):
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    O, lse = torch.full_like(x.Q, 7.0), torch.full(x.Q.shape[:3], 7.0, device="cuda")
    got = fbd.attn_paged(x.Q, x.cache, x.lens, x.cu, O=O, lse=lse, causal=causal, window=window, scale=scale,
                         max_new=max(x.new + [0]) if max_new is None else max_new, **kw)
    fbd.attn_device_status()
    assert got[0] is O and got[1] is lse
    if not check:
        return O, lse
    inside = torch.zeros(x.rows, dtype=torch.bool, device="cuda")
    for b, (o, L) in enumerate(R.attention(x, causal, window, scale or None, sums)):
        r, rows = x.place(b)
        inside[r, rows] = True
        within(O[r, :, rows], o, f"O of sequence {b}")
        within(lse[r, :, rows], L, f"lse of sequence {b}")
    out = ~inside[:, None].expand(x.rows[0], x.H, x.rows[1])
    assert (O[out] == 7.0).all() and (lse[out] == 7.0).all()  # rows of no sequence
    return O, lse


def batch(new, lens, page=16, heads=(2, 2), d=64, dtype="bf16", **kw):
    import paged_reference as R
    return R.Batch(new, lens, page, heads, d, dt(dtype), **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 17, 63, 64, 65, 127, 128, 129, 300])
def test_one_chunk(n, d, dtype):
    for before in (0, 1, 130):
        attend(batch([n], [n + before], d=d, dtype=dtype))
    attend(batch([n], [n + 90], d=d, dtype=dtype), causal=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("heads", [(1, 1), (2, 1), (6, 2), (8, 1), (5, 1), (16, 2), (48, 1)])
def test_one_token_each(heads, d, dtype):
    attend(batch([1] * 6, [1, 2, 16, 300, 77, 1000], heads=heads, d=d, dtype=dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new,lens,page,heads,window,causal", [
    ([5, 0, 1, 200, 16], [40, 9, 1, 500, 700], 16, (4, 2), 0, True),
    ([5, 0, 1, 200, 16], [40, 9, 1, 500, 700], 48, (6, 2), 0, False),
    ([300, 1, 1], [300, 2000, 900], 64, (3, 1), 0, True),
    ([129, 257], [129, 1000], 128, (2, 2), 100, True),
    ([64, 1, 1], [600, 600, 3], 256, (8, 2), 1, True),
    ([3, 2, 4], [900, 700, 4], 16, (12, 4), 130, True),
    ([400], [3000], 80, (7, 1), 1000, True),
    ([1] * 40, list(range(1, 41)), 16, (2, 1), 0, True),
    ([33] * 9, [33 + 20 * k for k in range(9)], 32, (10, 2), 0, True),
])
def test_ragged_batches(new, lens, page, heads, window, causal, dtype):
    for d, token_major in ((64, False), (128, True)):
        attend(batch(new, lens, page, heads, d, dtype, behind=5, token_major=token_major), causal=causal, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [(128, 1), (131, 1), (130, 1), (200, 2)])
def test_many_heads_to_a_key_head(heads, dtype):
    attend(batch([3, 1], [50, 200], heads=heads, d=64, dtype=dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_batch_that_is_not_packed(dtype):
    attend(batch([9] * 4, [9, 30, 200, 11], heads=(4, 2), dtype=dtype, packed=False))
    attend(batch([1] * 4, [9, 30, 200, 1], heads=(4, 2), dtype=dtype, packed=False, d=128))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_hint_of_new_tokens_left_out_or_wrong(dtype):
    """max_new chooses the kernel; none given, too large or too small a one gives the same values."""
    x = batch([5, 1, 40], [50, 600, 300], heads=(4, 1), d=128, dtype=dtype)
    for hint in (0, 1, 3, 1000):
        attend(x, max_new=hint)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scales(dtype):
    for scale in (0.02, 0.5):
        attend(batch([70, 1], [300, 400], d=64, dtype=dtype), scale=scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_see_nothing(dtype):
    """An empty sequence, one with fewer keys than new tokens, pages given up: O = 0 and lse = -inf."""
    torch = _t()
    attend(batch([2, 3], [0, 0], dtype=dtype))
    attend(batch([1, 1, 1], [0, 5, 0], dtype=dtype, heads=(4, 1)))
    attend(batch([20, 3], [7, 40], dtype=dtype))
    attend(batch([3], [0], dtype=dtype), causal=False)
    for n in (1, 50):
        x = batch([n, 1], [n + 300, 200], heads=(4, 2), dtype=dtype, d=128)
        x.table[0, 0] = -1
        x.table[0, 5] = x.K.shape[0]
        x.table[1, :] = -1
        attend(x)
        attend(x, window=60)
        attend(x, causal=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_what_a_token_does_not_see_has_no_part(d, bad, dtype):
    """Rows of the cache behind the last key, before a window, of a later token: whatever they hold."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    for new, lens, window, spoil in (([1, 1], [75, 140], 0, "behind"), ([40, 1], [75, 300], 0, "behind"),
                                     ([1, 1], [75, 140], 50, "before"), ([40, 200], [175, 300], 64, "before"),
                                     ([40, 3], [75, 30], 0, "last"), ([150, 3], [475, 30], 0, "last"),
                                     ([300, 2], [300, 2], 0, "last")):
        x = batch(new, lens, heads=(4, 2), d=d, dtype=dtype)
        clean, _ = attend(x, window=window)
        clean = clean.clone()
        for b, n in enumerate(lens):
            where = []
            if spoil == "behind":
                where = range(n, (n + 15) // 16 * 16)
            elif spoil == "before":
                where = range(0, max(0, n - new[b] - window + 1))
            else:
                where = [n - 1]  # seen by the last token alone
            for j in where:
                x.K[x.table[b, j // 16], :, j % 16] = bad
                x.V[x.table[b, j // 16], :, j % 16] = bad
        got, lse = attend(x, window=window, check=False)
        for b in range(len(new)):
            r, rows = x.place(b)
            see = slice(rows.start, rows.stop - (spoil == "last"))
            assert torch.equal(got[r, :, see], clean[r, :, see]), (new, spoil, b)
            if spoil == "last":
                assert not torch.isfinite(got[r, :, rows.stop - 1]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_same_bits_on_every_call(dtype):
    torch = _t()
    x = batch([90, 1, 5], [700, 2000, 5], heads=(4, 1), d=128, dtype=dtype)
    a = [t.clone() for t in attend(x)]
    for _ in range(3):
        assert all(torch.equal(u, v) for u, v in zip(a, attend(x)))


# ---------------------------------------------------------------------- a run of them together
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_prompt_and_its_next_tokens(dtype):
    """A layer's serving run: a prompt in two chunks, then three single tokens, against attention over
    the whole sequence at once (attn_qk_norm, attn_fwd): norm, rotary, cache and attention together."""
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    B, N, H, Hkv, d, page = 2, 203, 4, 2, 64, 32
    qkv = randn(B, N, H + 2 * Hkv, d, dtype=dt(dtype))
    q, k, v = (t.transpose(1, 2) for t in qkv.split([H, Hkv, Hkv], 2))
    wq, wk = (1 + 0.1 * randn(d, dtype=torch.float32, seed=s) for s in (1, 2))
    _, freq, axis = tables(1, 1, d, 1)
    pos = torch.arange(N, device="cuda", dtype=torch.int32)[None]
    qn, kn = fbd.attn_qk_norm((q, k), (wq, wk), pos, freq, axis)
    whole, lse = fbd.attn_fwd(qn, kn, v.contiguous())
    width = (N + page - 1) // page
    K = torch.full((B * width, Hkv, page, d), float("nan"), dtype=q.dtype, device="cuda")
    V = torch.full_like(K, float("inf"))
    table = torch.randperm(B * width, device="cuda").int().view(B, width)
    tol = (2 * 2.0 ** -8 if dtype == "bf16" else 0.0) + 2 * R.FP32  # both sides round P and O, and the keys alike
    done = 0
    for n in (120, 80, 1, 1, 1):
        s = slice(done, done + n)
        done += n
        lens = torch.full((B,), done, dtype=torch.int32, device="cuda")
        qq = fbd.attn_cache_append(k[:, :, s], v[:, :, s], (K, V, table), lens, Q=q[:, :, s], weights=(wq, wk), freq=freq, axis=axis)
        assert torch.equal(qq, qn[:, :, s])
        O, L = fbd.attn_paged(qq, (K, V, table), lens)
        fbd.attn_device_status()
        assert (L - lse[:, :, s]).abs().max() <= 2 * R.FP32 * (1 + lse.abs().max())
        mag = v.double().abs().max()  # a weighted mean of V's rows
        assert (O.double() - whole[:, :, s].double()).abs().max() <= tol * mag + 2 * R.half_step(q.dtype) * mag
