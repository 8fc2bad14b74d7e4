"""Appends and normed heads of the sizes that a prompt or a training batch has, where a block takes several heads and
token after token: against the plain references at once, every token of them.  Bounds: tests/paged_reference.py."""
import random

import pytest

from test_gpu_paged import _lib, _t, batch, dt, randn, tables, within  # noqa: F401

pytestmark = pytest.mark.gpu


def append_all(new, lens, page, heads, d, dtype, packed=True, normed=True, axes=0, paired="half", in_place=False, with_q=True, **kw):
    """One append, every key, value and query of it compared, and all that it has to leave alone.  axes: positions given
    (0: the tokens' own)."""
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    x = batch(new, lens, page, heads, d, dtype, packed=packed, **kw)
    B, N = x.rows
    qkv = x.randn(B, N, x.H + 2 * x.Hkv, d)
    q, k, v = (t.transpose(1, 2) for t in qkv.split([x.H, x.Hkv, x.Hkv], 2))
    ws = [1 + 0.2 * randn(d, dtype=torch.float32, seed=s) for s in (5, 6)] if normed else None
    # of each row: its sequence (-1: none) and its position there
    seq = torch.full((B, N), -1, dtype=torch.int64, device="cuda")
    at = torch.zeros((B, N), dtype=torch.int64, device="cuda")
    for b, n in enumerate(new):
        r, rows = x.place(b)
        seq[r, rows] = b
        at[r, rows] = max(lens[b], 0) - n + torch.arange(n, device="cuda")
    pos, freq, axis = tables(B, N, d, max(axes, 1))
    cs = R.cos_sin(pos if axes else at[None], freq, axis)
    K0, V0, q0 = x.K.clone(), x.V.clone(), q.clone()
    out = None if not with_q else q if in_place else torch.full((B, N, x.H, d), 7.0, dtype=q.dtype, device="cuda").transpose(1, 2)
    got = fbd.attn_cache_append(k, v, x.cache, x.lens, x.cu, Q=q if with_q else None, Q_out=out, weights=ws,
                                pos=pos if axes else None, freq=freq, axis=axis, paired=paired)
    fbd.attn_device_status()
    assert got is out

    def made(t, w):
        if normed:
            return R.norm(t, w, cs, paired)
        y, mag = R.turn(t.double(), cs, paired)
        return y, R.NORM * mag + R.half_step(t.dtype) * y.abs()

    inside = seq >= 0
    entry = at.clamp(min=0) // page
    p = x.table[seq.clamp(min=0), entry.clamp(max=x.width - 1)].long()
    put = inside & (at >= 0) & (entry < x.width) & (p >= 0) & (p < x.K.shape[0])
    slot = at.clamp(min=0) % page
    assert put.any()
    rows = lambda t: t.transpose(1, 2)[put]  # noqa: E731  [tokens, heads, d]
    y, tol = made(k, ws[1] if normed else None)
    within(x.K[p[put], :, slot[put]], (rows(y), rows(tol)), "keys")
    assert torch.equal(x.V[p[put], :, slot[put]], rows(v))
    hit = torch.zeros(x.K.shape[0], page, dtype=torch.bool, device="cuda")
    hit[p[put], slot[put]] = True
    away = ~hit[:, None, :, None].expand(x.K.shape)
    assert torch.equal(x.K[away], K0[away]) and torch.equal(x.V[away], V0[away])  # nothing else is written
    if with_q:
        y, tol = made(q0, ws[0] if normed else None)
        t = out.transpose(1, 2)
        within(t[inside], (y.transpose(1, 2)[inside], tol.transpose(1, 2)[inside]), "queries")
        rest = q0.transpose(1, 2)[~inside] if in_place else torch.full_like(t[~inside], 7.0)
        assert torch.equal(t[~inside], rest)  # rows of no sequence


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("normed,axes,paired,in_place", [(True, 0, "half", False), (True, 2, "neighbour", True),
                                                         (False, 0, "neighbour", True), (False, 3, "half", False)])
def test_prompts(normed, axes, paired, in_place, dtype):
    new = [2100, 0, 3990, 517, 1, 1460, 3333]
    append_all(new, [n + c for n, c in zip(new, (0, 40, 300, 0, 77, 13, 260))], 64, (16, 4), 128, dtype, normed=normed, axes=axes,
               paired=paired, in_place=in_place, behind=5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,heads", [(32, (12, 12)), (64, (12, 4)), (96, (6, 2)), (256, (8, 1))])
def test_prompts_of_every_head_dim(d, heads, dtype):
    new = [1900, 731, 4001]
    append_all(new, [n + 9 for n in new], 48, heads, d, dtype, token_major=True)
    append_all([1500] * 3, [1500, 1777, 2000], 32, heads, d, dtype, packed=False, axes=2, in_place=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B", [511, 512, 513, 600, 3000])
def test_appends_of_many_sequences(B, dtype):
    """More sequences than a block holds the lengths of, empty ones among them, and rows behind the last."""
    rng = random.Random(B)
    new = [rng.choice([0, 1, 1, 2, 9]) for _ in range(B)]
    new[0] = new[-1] = 0
    lens = [n + rng.randint(0, 60) for n in new]
    append_all(new, lens, 16, (4, 2), 64, dtype, behind=7)
    append_all(new, lens, 16, (4, 2), 64, dtype, behind=7, axes=2, with_q=False)
    append_all([1] * B, [1 + i % 50 for i in range(B)], 16, (4, 2), 64, dtype, packed=False, in_place=True)
    append_all([3] * B, [3 + i % 50 for i in range(B)], 16, (4, 2), 64, dtype, packed=False, axes=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts_outside_the_table_or_the_cache(dtype):
    """Long runs of tokens before the first key, behind the table or on pages given up: their queries alone are made."""
    append_all([2000, 3000], [900, 3500], 64, (8, 2), 128, dtype, width=40)
    append_all([2000] * 2, [-5, 3500], 64, (8, 2), 128, dtype, width=40, packed=False)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("paired", ["half", "neighbour"])
@pytest.mark.parametrize("B,N,HQ,HK,d", [(4, 8192, 12, 12, 64), (3, 9999, 6, 2, 96), (30001, 1, 4, 1, 32), (1, 20011, 5, 5, 128), (2, 7001, 8, 3, 256)])
def test_normed_heads_of_many_tokens(B, N, HQ, HK, d, paired, dtype):
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    qk = randn(B, N, HQ + HK, d, dtype=dt(dtype))
    xs = [t.transpose(1, 2) for t in qk.split([HQ, HK], 2)]
    ws = [1 + 0.3 * randn(d, dtype=torch.float32, seed=k) for k in (1, 2)]
    pos, freq, axis = tables(B, N, d, 2)
    cs = R.cos_sin(pos, freq, axis)
    ys = fbd.attn_qk_norm(xs, ws, pos, freq, axis, paired=paired)
    fbd.attn_device_status()
    for k, (x, w) in enumerate(zip(xs, ws)):
        within(ys[k], R.norm(x, w, cs, paired), f"y[{k}]")
    keep = [y.clone() for y in ys]
    fbd.attn_qk_norm(xs, ws, pos, freq, axis, outs=xs, paired=paired)  # in place
    assert all(torch.equal(a, b) for a, b in zip(xs, keep))
