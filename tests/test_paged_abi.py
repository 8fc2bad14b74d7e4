"""Host-side checks of the normed heads, the append and the attention over a paged cache that need no GPU:
bad arguments are refused synchronously (fake pointers are never dereferenced) and the binding refuses
tensors of the wrong shape, type or place."""
import ctypes

import pytest

import __graft_entry__

__graft_entry__.build()
import fwd_bwd_double_gb300 as fbd  # noqa: E402
from fwd_bwd_double_gb300 import AttnDesc, Cache, FbdError, NewTokens, NormGrad, NormTensor, RopeDesc, lib  # noqa: E402

OK, INVALID, UNSUP, ALIGN, WS = 0, 1, 2, 3, 4
FAKE = 1 << 40


def at(k):
    return FAKE + k * (1 << 34)


def p(x):
    return ctypes.c_void_p(x)


# ------------------------------------------------------------------------------ normed heads
HEADS, B, N, D = 4, 2, 8, 64
DENSE = (HEADS * N * D, N * D, D)


def rope_desc(d=D, dtype=1, paired=0, inverse=0, axes=2, pbs=N, B=B, N=N):
    return RopeDesc(B, N, d, axes, dtype, paired, inverse, pbs)


def norm(x=at(0), y=at(1), w=at(2), heads=HEADS, xs=DENSE, ys=DENSE, pos=at(3), freq=at(4), axis=at(5), eps=1e-6, count=1,
         tensors=True, **kw):
    t = (NormTensor * 4)()
    for k in range(4):
        t[k].x, t[k].y, t[k].w, t[k].heads = x, y and y + k * (1 << 32), w, heads
        t[k].x_stride[:], t[k].y_stride[:] = xs, ys
    return lib.attn_qk_norm(ctypes.byref(rope_desc(**kw)), t if tensors else None, count, eps, p(pos), p(freq), p(axis), None)


def norm_bwd(x=at(0), dy=at(1), dx=at(2), w=at(3), dw=at(4), heads=HEADS, xs=DENSE, dys=DENSE, dxs=DENSE, pos=at(5), freq=at(6),
             axis=at(7), eps=1e-6, ws=at(8), nbytes=None, count=1, **kw):
    t = (NormGrad * 4)()
    for k in range(4):
        t[k].x, t[k].dy, t[k].dx, t[k].w, t[k].heads = x, dy, dx and dx + k * (1 << 32), w, heads
        t[k].dw = dw and dw + k * 4096
        t[k].x_stride[:], t[k].dy_stride[:], t[k].dx_stride[:] = xs, dys, dxs
    d = rope_desc(**kw)
    need = lib.attn_qk_norm_bwd_workspace_bytes(ctypes.byref(d), t, count) if nbytes is None else nbytes
    return lib.attn_qk_norm_bwd(ctypes.byref(d), t, count, eps, p(pos), p(freq), p(axis), p(ws), need, None)


SHARED = [
    (dict(d=48), UNSUP), (dict(dtype=3), UNSUP), (dict(paired=2), UNSUP), (dict(inverse=1), UNSUP), (dict(axes=0), INVALID),
    (dict(axes=65), INVALID), (dict(pbs=3), INVALID), (dict(B=-1), INVALID), (dict(N=1 << 31), INVALID), (dict(count=0), INVALID),
    (dict(count=5), INVALID), (dict(heads=-1), INVALID), (dict(heads=70000), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(x=0), INVALID), (dict(x=at(0) + 8), ALIGN),
    (dict(xs=(2048, 516, 64)), ALIGN), (dict(xs=(2048, -512, 64)), INVALID), (dict(w=at(9) + 2), ALIGN),
    (dict(pos=0), INVALID), (dict(freq=0), INVALID), (dict(axis=0), INVALID), (dict(pos=at(9) + 2), ALIGN),
]


@pytest.mark.parametrize("kw,code", SHARED)
def test_norm_refuses(kw, code):
    assert norm(**kw) == code and lib.attn_last_error()
    assert norm_bwd(**kw) == code and lib.attn_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(y=0), INVALID), (dict(y=at(1) + 8), ALIGN), (dict(ys=(2048, 0, 64)), INVALID), (dict(ys=(2048, 512, 32)), INVALID),
    (dict(y=at(0) + 64), INVALID), (dict(y=at(3)), INVALID), (dict(y=at(2) - 64), INVALID), (dict(tensors=False), INVALID),
    (dict(y=at(0), ys=(DENSE[0], D, HEADS * D)), INVALID), (dict(count=2, x=at(1), y=at(1)), INVALID),
])
def test_norm_refuses_outputs(kw, code):
    assert norm(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(dx=0), INVALID), (dict(dy=0), INVALID), (dict(dx=at(2) + 8), ALIGN), (dict(dys=(2048, 512, 60)), ALIGN),
    (dict(dxs=(2048, 512, 32)), INVALID), (dict(dx=at(0) + 64), INVALID), (dict(dx=at(1) + 64), INVALID),
    (dict(dw=at(3)), INVALID), (dict(dw=at(2)), INVALID), (dict(dw=at(0)), INVALID), (dict(dw=at(9) + 1), ALIGN),
    (dict(ws=0), WS), (dict(nbytes=64), WS), (dict(ws=at(8) + 4), ALIGN), (dict(ws=at(2)), INVALID), (dict(ws=at(4)), INVALID),
])
def test_norm_bwd_refuses_outputs(kw, code):
    assert norm_bwd(**kw) == code


def test_norm_empty():
    for kw in (dict(B=0), dict(N=0, pbs=0), dict(heads=0)):
        assert norm(x=0, y=0, w=0, pos=0, freq=0, axis=0, **kw) == OK
        assert norm_bwd(x=0, dy=0, dx=0, w=0, dw=0, pos=0, freq=0, axis=0, ws=0, **kw) == OK
    assert lib.attn_qk_norm(None, None, 1, 1e-6, None, None, None, None) == INVALID
    assert lib.attn_qk_norm_bwd(None, None, 1, 1e-6, None, None, None, None, 0, None) == INVALID
    assert lib.attn_qk_norm_bwd_workspace_bytes(None, None, 1) == 0


# ------------------------------------------------------------------------- cache and attention
PAGES, PAGE, WIDTH, SEQS, T, H, HKV = 10, 16, 5, 3, 20, 8, 2


def desc(B=SEQS, H=H, N=T, d=D, scale=0.0, causal=1, dtype=1, group=H // HKV, window=0, lo=None, hi=None):
    return AttnDesc(B, H, N, d, scale, causal, dtype, group, window, lo, hi)


def cache(K=at(10), V=at(11), table=at(12), pages=PAGES, page_size=PAGE, width=WIDTH, ks=(HKV * PAGE * D, PAGE * D, D), vs=None):
    c = Cache()
    c.K, c.V, c.table, c.pages, c.page_size, c.width = K, V, table, pages, page_size, width
    c.k_stride[:], c.v_stride[:] = ks, vs or ks
    return c


QS = (0, D, H * D)  # packed tokens, token by token


def paged(Q=at(0), O=at(1), lse=at(2), cu=at(3), lens=at(4), ws=at(5), nbytes=None, qs=QS, os=QS, max_new=0, c=None, d=None, **kw):
    dsc = d or desc(**{k: kw.pop(k) for k in list(kw) if k in ("B", "H", "N", "d_", "scale", "causal", "dtype", "group", "window", "lo", "hi")})
    need = lib.attn_paged_workspace_bytes(ctypes.byref(dsc), max_new) if nbytes is None else nbytes
    S = ctypes.c_int64 * 3
    return lib.attn_paged(ctypes.byref(dsc), p(Q), S(*qs) if qs else None, ctypes.byref(c or cache(**kw)), p(cu), p(lens), max_new, p(O),
                          S(*os) if os else None, p(lse), p(ws), need, None)


def append(K=at(0), V=at(1), Q=at(2), Q_out=at(3), cu=at(4), lens=at(5), kw_=at(6), qw=at(7), pos=0, freq=at(8), axis=at(9), pbs=0,
           axes=1, paired=0, normed=1, eps=1e-6, ks=(0, D, HKV * D), qs=QS, qos=QS, dsc=None, c=None, **kw):
    t = NewTokens()
    t.K, t.V, t.Q, t.Q_out, t.k_weight, t.q_weight, t.pos, t.freq, t.axis = K, V, Q, Q_out, kw_, qw, pos, freq, axis
    t.k_stride[:], t.v_stride[:], t.q_stride[:], t.q_out_stride[:] = ks, ks, qs, qos
    t.pos_batch_stride, t.axes, t.paired, t.normed, t.eps = pbs, axes, paired, normed, eps
    return lib.attn_cache_append(ctypes.byref(dsc or desc()), ctypes.byref(t), ctypes.byref(c or cache(**kw)), p(cu), p(lens), None)


@pytest.mark.parametrize("dsc,code", [
    (dict(d=48), UNSUP), (dict(dtype=4), UNSUP), (dict(causal=2), UNSUP), (dict(B=-1), INVALID), (dict(N=-1), INVALID),
    (dict(H=9), INVALID), (dict(group=3), INVALID), (dict(window=-1), INVALID), (dict(window=4, causal=0), UNSUP),
    (dict(scale=float("nan")), INVALID), (dict(scale=-1.0), INVALID), (dict(N=1 << 31), INVALID), (dict(B=1 << 26), INVALID),
    (dict(lo=at(13), hi=at(14)), UNSUP), (dict(lo=at(13)), INVALID), (dict(H=70000, group=70000), INVALID),
])
def test_paged_refuses_bad_descriptors(dsc, code):
    assert paged(d=desc(**dsc), nbytes=1 << 40) == code and lib.attn_last_error()
    assert append(dsc=desc(**dsc)) == code
    assert lib.attn_paged_workspace_bytes(ctypes.byref(desc(**dsc)), 0) == 0


CACHES = [
    (dict(page_size=8), UNSUP), (dict(page_size=24), UNSUP), (dict(page_size=0), UNSUP), (dict(page_size=-16), UNSUP),
    (dict(page_size=1 << 21), UNSUP), (dict(pages=-1), INVALID), (dict(pages=1 << 31), INVALID), (dict(width=-1), INVALID),
    (dict(width=1 << 27), INVALID), (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(K=at(10) + 8), ALIGN), (dict(table=0), INVALID),
    (dict(table=at(12) + 2), ALIGN), (dict(ks=(2048, 1024, 60)), ALIGN), (dict(ks=(2048, 0, 64)), INVALID),
    (dict(ks=(2048, -1024, 64)), INVALID), (dict(lens=0), INVALID), (dict(lens=at(13) + 2), ALIGN), (dict(cu=at(14) + 2), ALIGN),
]


@pytest.mark.parametrize("kw,code", CACHES)
def test_paged_refuses_bad_caches(kw, code):
    assert paged(**kw) == code and lib.attn_last_error()
    own = {k: v for k, v in kw.items() if k in ("lens", "cu")}
    assert append(c=cache(**{k: v for k, v in kw.items() if k not in own}), **own) == code and lib.attn_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(Q=0), INVALID), (dict(O=0), INVALID), (dict(Q=at(0) + 8), ALIGN), (dict(O=at(1) + 8), ALIGN), (dict(lse=at(2) + 2), ALIGN),
    (dict(qs=None), INVALID), (dict(os=None), INVALID), (dict(qs=(0, 0, 512)), INVALID), (dict(qs=(0, 64, 516)), ALIGN),
    (dict(os=(0, 32, 512)), INVALID), (dict(ws=0), WS), (dict(nbytes=100), WS), (dict(ws=at(5) + 8), ALIGN), (dict(max_new=-1), INVALID),
    (dict(O=at(0)), INVALID), (dict(O=at(10)), INVALID), (dict(O=at(11) + 1024), INVALID), (dict(O=at(12)), INVALID),
    (dict(O=at(3)), INVALID), (dict(O=at(4)), INVALID), (dict(lse=at(1)), INVALID), (dict(lse=at(0)), INVALID), (dict(ws=at(0)), INVALID),
    (dict(ws=at(1)), INVALID), (dict(ws=at(2)), INVALID), (dict(ws=at(10)), INVALID),
])
def test_paged_refuses(kw, code):
    assert paged(**kw) == code and lib.attn_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(K=0), INVALID), (dict(V=0), INVALID), (dict(V=at(1) + 8), ALIGN), (dict(Q=0), INVALID), (dict(Q_out=0), INVALID),
    (dict(ks=(0, 64, 124)), ALIGN), (dict(qos=(0, 32, 512)), INVALID), (dict(normed=2), UNSUP), (dict(paired=3), UNSUP),
    (dict(eps=-1.0), INVALID), (dict(freq=0), INVALID), (dict(axis=0), INVALID), (dict(freq=at(8) + 2), ALIGN), (dict(axes=2), INVALID),
    (dict(pos=at(13), axes=0), INVALID), (dict(pos=at(13) + 2), ALIGN), (dict(pos=at(13), pbs=3), INVALID), (dict(kw_=at(6) + 2), ALIGN),
    (dict(qw=at(7) + 2), ALIGN), (dict(Q_out=at(2) + 64), INVALID), (dict(Q_out=at(0)), INVALID), (dict(Q_out=at(10)), INVALID),
    (dict(Q_out=at(12)), INVALID), (dict(Q_out=at(5)), INVALID), (dict(Q_out=at(8)), INVALID), (dict(Q_out=at(6)), INVALID),
    (dict(c="K=V"), INVALID), (dict(c="K over new"), INVALID), (dict(c="gaps"), INVALID), (dict(c="V over table"), INVALID),
])
def test_append_refuses(kw, code):
    if "c" in kw:
        kw = dict(c={"K=V": cache(K=at(11)), "K over new": cache(K=at(0)), "gaps": cache(ks=(2048, 512, 64)),
                     "V over table": cache(V=at(12))}[kw["c"]])
    assert append(**kw) == code and lib.attn_last_error()


def test_paged_workspace_and_empty_calls():
    for dtype in (0, 1):
        for d in (32, 64, 96, 128, 256):
            for hint in (0, 1, 5, 1 << 40):
                n = lib.attn_paged_workspace_bytes(ctypes.byref(desc(d=d, dtype=dtype)), hint)
                assert 0 < n < 1 << 28
                assert paged(d=desc(d=d, dtype=dtype), max_new=hint, nbytes=n - 1, qs=(0, d, H * d), os=(0, d, H * d),
                             c=cache(ks=(HKV * PAGE * d, PAGE * d, d))) == WS
    assert lib.attn_paged_workspace_bytes(None, 0) == 0
    for kw in (dict(B=0), dict(H=0, group=0), dict(N=0)):
        assert paged(Q=0, O=0, lse=0, cu=0, lens=0, ws=0, nbytes=0, K=0, V=0, table=0, **kw) == OK
        assert append(K=0, V=0, Q=0, Q_out=0, cu=0, lens=0, dsc=desc(**kw)) == OK
    assert lib.attn_paged(None, None, None, None, None, None, 0, None, None, None, None, 0, None) == INVALID
    assert lib.attn_cache_append(None, None, None, None, None, None) == INVALID
    assert lib.attn_cache_append(ctypes.byref(desc()), None, None, None, None, None) == INVALID


def test_binding_refuses_shapes_types_and_places():
    import torch
    z = torch.zeros
    Q, k, v = z(1, 4, 6, 64), z(1, 2, 6, 64), z(1, 2, 6, 64)
    K, V, table = z(5, 2, 16, 64), z(5, 2, 16, 64), z(3, 4, dtype=torch.int32)
    lens, cu = z(3, dtype=torch.int32), z(4, dtype=torch.int32)
    c = (K, V, table)
    freq, axis, w = z(32), z(32, dtype=torch.int32), z(64)
    pos = z(1, 6, dtype=torch.int32)
    P, A = fbd.attn_paged, fbd.attn_cache_append
    bad = [lambda: P(Q, c, lens, cu),                                   # on the CPU
           lambda: P(Q, c, lens), lambda: P(Q[0], c, lens, cu), lambda: P(None, c, lens, cu), lambda: P(Q, None, lens, cu),
           lambda: P(Q, (K, V), lens, cu), lambda: P(Q, (K, None, table), lens, cu), lambda: P(Q, (K, V, None), lens, cu),
           lambda: P(Q, (K[0], V, table), lens, cu), lambda: P(Q, (K, V[:4], table), lens, cu), lambda: P(Q, (K, V.bfloat16(), table), lens, cu),
           lambda: P(Q, (K, V, table.long()), lens, cu), lambda: P(Q, (K, V, table[:2]), lens, cu), lambda: P(Q, (K, V, table[0]), lens, cu),
           lambda: P(Q, c, None, cu), lambda: P(Q, c, lens.long(), cu), lambda: P(Q, c, lens[:2], cu), lambda: P(Q, c, lens, cu[:3]),
           lambda: P(Q, c, lens, cu.long()), lambda: P(Q[:, :3], c, lens, cu), lambda: P(Q[..., :32], c, lens, cu),
           lambda: P(Q.half(), c, lens, cu), lambda: P(Q, c, lens, cu, O=Q[:, :, :3]), lambda: P(Q, c, lens, cu, lse=z(1, 4, 5)),
           lambda: P(Q.transpose(2, 3), (z(5, 2, 16, 6), z(5, 2, 16, 6), table), lens, cu), lambda: P(Q, c, lens[None], cu),
           lambda: P(Q, c, lens, cu, window=-1), lambda: P(Q, c, lens, cu, causal=False, window=3), lambda: P(Q, (K[:, :0], V[:, :0], table), lens, cu),
           lambda: A(k, v, c, lens, cu),                                # on the CPU
           lambda: A(None, v, c, lens, cu), lambda: A(k, None, c, lens, cu), lambda: A(k, v[:, :, :2], c, lens, cu),
           lambda: A(k, v, c, lens), lambda: A(k, v, c, lens, cu, Q=Q[:, :3]), lambda: A(k, v, c, lens, cu, Q_out=Q),
           lambda: A(k, v, c, lens, cu, Q=Q, Q_out=Q[:, :, :2]), lambda: A(k, v, c, lens, cu, weights=w), lambda: A(k, v, c, lens, cu, weights=(w,)),
           lambda: A(k, v, c, lens, cu, weights=(w, w.double())), lambda: A(k, v, c, lens, cu, weights=(w, w[:3])),
           lambda: A(k, v, c, lens, cu, freq=freq), lambda: A(k, v, c, lens, cu, axis=axis), lambda: A(k, v, c, lens, cu, pos=pos),
           lambda: A(k, v, c, lens, cu, freq=freq, axis=axis.long()), lambda: A(k, v, c, lens, cu, freq=freq[:3], axis=axis),
           lambda: A(k, v, c, lens, cu, pos=pos[:, :2], freq=freq, axis=axis), lambda: A(k, v, c, lens, cu, paired="x"),
           lambda: A(k[:, :1], v[:, :1], c, lens, cu), lambda: A(k.bfloat16(), v, c, lens, cu)]
    n, g = fbd.attn_qk_norm, fbd.attn_qk_norm_bwd
    bad += [lambda: n(Q),                                               # on the CPU
            lambda: n(None), lambda: n([]), lambda: n([Q] * 5), lambda: n(Q[0]), lambda: n((Q, None)), lambda: n(Q, w.double()), lambda: n(Q, w[:3]),
            lambda: n((Q, k), (w,)), lambda: n((Q, k), w), lambda: n(Q, w, pos), lambda: n(Q, w, None, freq, axis), lambda: n(Q, w, pos, freq),
            lambda: n(Q, w, pos.long(), freq, axis), lambda: n(Q, w, pos, freq, axis, paired="x"), lambda: n(Q, w, outs=[Q, Q]),
            lambda: n(Q, w, outs=k), lambda: n((Q, k.bfloat16())), lambda: n(Q.half()), lambda: n(Q, eps=-1.0),
            lambda: g(Q, Q), lambda: g(Q, None), lambda: g(Q, k), lambda: g((Q, k), (Q,)), lambda: g(Q, Q.bfloat16()), lambda: g(Q, Q, w[:3]),
            lambda: g(Q, Q, w, dweights=w[:3]), lambda: g(Q, Q, w, dxs=k), lambda: g(Q, Q, w, workspace=z(2, 2).t())]
    for i, f in enumerate(bad):
        with pytest.raises(FbdError):
            f()
            raise AssertionError(f"case {i} was accepted")
    for s in (0, 1 << 40):  # host tensors given a stream
        with pytest.raises(FbdError):
            P(Q, c, lens, cu, stream=s)


def test_window_and_hint_past_32_bits():
    """A window as wide as the cache or wider is none; the descriptor's field has 32 bits."""
    import torch
    Q, K, table = torch.zeros(1, 4, 6, 64), torch.zeros(5, 2, 16, 64), torch.zeros(3, 4, dtype=torch.int32)
    lens, cu = torch.zeros(3, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for window, hint in ((1 << 40, 1 << 40), ((1 << 32) + 5, 7)):
        with pytest.raises(FbdError, match="one CUDA device"):  # past every other check
            fbd.attn_paged(Q, (K, K.clone(), table), lens, cu, window=window, max_new=hint)


def test_tokens_at_the_end_of_the_index_range():
    """Token counts whose last tile would end behind 2^31 are refused; the most that are taken pass the descriptor."""
    for n, code in (((1 << 31) - 1, INVALID), ((1 << 31) - 4095, INVALID), ((1 << 31) - 4096, WS)):
        d = desc(B=1, H=1, N=n, group=1)
        assert paged(d=d, nbytes=0, qs=(0, 0, D), os=(0, 0, D), Q=1 << 50, O=1 << 51, lse=0) == code
        assert (lib.attn_paged_workspace_bytes(ctypes.byref(d), 0) > 0) == (code == WS)
        if code == INVALID:
            assert append(dsc=d) == code
