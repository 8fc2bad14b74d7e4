"""Host-side checks of the differential attention and rotary entry points that need no GPU:
bad arguments are refused synchronously (fake pointers are never dereferenced) and the
binding refuses tensors of the wrong shape, type or place."""
import ctypes

import pytest

import __graft_entry__

__graft_entry__.build()
import fwd_bwd_double_gb300 as fbd  # noqa: E402
from fwd_bwd_double_gb300 import AttnDesc, FbdError, RopeDesc, RopeTensor, lib  # noqa: E402

OK, INVALID, UNSUP, ALIGN, WS = 0, 1, 2, 3, 4
FAKE = 1 << 40


def desc(B=1, H=2, N=64, d=64, scale=0.0, causal=1, dtype=1, group=0, window=0, lo=None, hi=None):
    return AttnDesc(B, H, N, d, scale, causal, dtype, group, window, lo, hi)


def ptrs(n):
    return [ctypes.c_void_p(FAKE + i * (1 << 32)) for i in range(n)]


def fwd(dsc, p=None):
    return lib.attn_diff_fwd(ctypes.byref(dsc), *(p or ptrs(7)), None)


def bwd(dsc, p=None, ws=None):
    p = p or ptrs(13)
    ws = lib.attn_diff_bwd_workspace_bytes(ctypes.byref(dsc)) if ws is None else ws
    return lib.attn_diff_bwd(ctypes.byref(dsc), *p, ws, None)


def decode(dsc, p=None, ws=None):
    p = p or ptrs(7)
    ws = lib.attn_diff_decode_workspace_bytes(ctypes.byref(dsc)) if ws is None else ws
    return lib.attn_diff_decode(ctypes.byref(dsc), *p, ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), UNSUP), (dict(d=128), UNSUP), (dict(d=16), UNSUP), (dict(dtype=5), UNSUP), (dict(causal=2), UNSUP),
    (dict(B=-1), INVALID), (dict(H=3, group=2), INVALID), (dict(window=-1), INVALID), (dict(scale=-1.0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(causal=0, window=4), UNSUP), (dict(N=1 << 31), INVALID),
    (dict(lo=FAKE), INVALID), (dict(B=1 << 15, H=1 << 15, N=1), INVALID), (dict(B=1 << 14, H=1 << 14, N=1), INVALID),
    (dict(B=1 << 10, H=1 << 10, N=(1 << 15) + 1), INVALID),
])
def test_refuses_bad_descriptors(kw, code):
    d = desc(**kw)
    assert fwd(d) == code and bwd(d, ws=1 << 50) == code and decode(d, ws=1 << 50) == code
    assert lib.attn_last_error()


def test_decode_refuses_full_and_document_masks():
    assert decode(desc(causal=0)) == UNSUP
    assert decode(desc(lo=FAKE, hi=FAKE + (1 << 36))) == UNSUP


@pytest.mark.parametrize("call,n,small", [(fwd, 7, (3,)), (bwd, 13, (3, 11)), (decode, 7, (3, 4))])
def test_refuses_null_and_misaligned_pointers(call, n, small):
    d = desc(N=4096)
    for i in range(n):
        if call is fwd and i == 5:  # O2 may be NULL
            continue
        p = ptrs(n)
        p[i] = ctypes.c_void_p(0)
        assert call(d, p) == (WS if i == n - 1 and call is not fwd else INVALID), i
        p = ptrs(n)
        p[i] = ctypes.c_void_p(FAKE + i * (1 << 32) + (2 if i in small else 8))
        assert call(d, p) == ALIGN, i


def test_refuses_overlaps():
    d = desc()
    for out, other in ((4, 0), (4, 2), (5, 1), (6, 4), (4, 3)):
        p = ptrs(7)
        p[out] = p[other]
        assert fwd(d, p) == INVALID, (out, other)
    for out, other in ((8, 0), (9, 8), (10, 2), (11, 3), (11, 6), (11, 10), (12, 5), (12, 3)):
        p = ptrs(13)
        p[out] = p[other]
        assert bwd(d, p) == INVALID, (out, other)
    for out, other in ((5, 0), (5, 1), (5, 3), (5, 4), (6, 5), (6, 2)):
        p = ptrs(7)
        p[out] = p[other]
        assert decode(desc(N=4096), p) == INVALID, (out, other)


def test_workspaces():
    d = desc(B=2, H=3, N=4096)
    for call, need in ((bwd, lib.attn_diff_bwd_workspace_bytes(ctypes.byref(d))),
                       (decode, lib.attn_diff_decode_workspace_bytes(ctypes.byref(d)))):
        assert need > 0
        assert call(d, ws=need - 1) == WS
    # more than 2^31 rows: 64-bit sizes
    big = desc(B=1, H=64, N=1 << 24)
    assert lib.attn_diff_bwd_workspace_bytes(ctypes.byref(big)) >= (1 << 24) * 64 * 16
    assert lib.attn_diff_bwd_workspace_bytes(None) == 0 and lib.attn_diff_decode_workspace_bytes(None) == 0


def test_empty_problems_touch_nothing():
    null = [ctypes.c_void_p(0)] * 13
    for kw in (dict(B=0), dict(H=0), dict(N=0)):
        assert fwd(desc(**kw), null[:7]) == OK
    assert bwd(desc(H=0), null) == OK
    assert decode(desc(B=0), null[:7]) == OK and decode(desc(H=0), null[:7]) == OK


def rope(B=2, N=8, d=64, axes=3, dtype=1, paired=0, inverse=0, pbs=None, heads=4, x=FAKE, y=FAKE + (1 << 36), xs=None,
         ys=None, count=1, ptr=None):
    dsc = RopeDesc(B, N, d, axes, dtype, paired, inverse, N if pbs is None else pbs)
    t = (RopeTensor * 4)()
    for k in range(4):
        t[k].x, t[k].y, t[k].heads = x, y + k * (1 << 32), heads
        t[k].x_stride[:] = xs or (heads * N * d, N * d, d)
        t[k].y_stride[:] = ys or (heads * N * d, N * d, d)
    return lib.attn_rope(ctypes.byref(dsc), t, count, *(ptr or ptrs(3)), None)


@pytest.mark.parametrize("kw,code", [
    (dict(d=48), UNSUP), (dict(d=0), UNSUP), (dict(dtype=3), UNSUP), (dict(paired=2), UNSUP), (dict(inverse=2), UNSUP),
    (dict(axes=0), INVALID), (dict(axes=65), INVALID), (dict(B=-1), INVALID), (dict(N=1 << 31), INVALID),
    (dict(pbs=5), INVALID), (dict(count=0), INVALID), (dict(count=5), INVALID), (dict(heads=-1), INVALID),
    (dict(heads=70000), INVALID), (dict(x=FAKE + 8), ALIGN), (dict(y=FAKE + 8), ALIGN), (dict(x=None), INVALID),
    (dict(xs=(2048, 516, 64)), ALIGN), (dict(xs=(2048, -512, 64)), INVALID), (dict(ys=(2048, 0, 64)), INVALID),
    (dict(ys=(2048, 512, 32)), INVALID), (dict(ys=(1024, 512, 64)), INVALID), (dict(y=FAKE + 1024), INVALID),
    (dict(xs=(2048, 512, 1 << 60)), INVALID),
])
def test_rope_refuses(kw, code):
    assert rope(**kw) == code
    assert lib.attn_last_error()


def test_rope_refuses_bad_tables():
    for k in range(3):
        p = ptrs(3)
        p[k] = ctypes.c_void_p(0)
        assert rope(ptr=p) == INVALID
        p[k] = ctypes.c_void_p(FAKE + 2)
        assert rope(ptr=p) == ALIGN


def test_rope_empty():
    for kw in (dict(B=0), dict(N=0), dict(heads=0)):
        assert rope(x=None, y=0, ptr=[ctypes.c_void_p(0)] * 3, **kw) == OK


def test_binding_refuses_shapes_types_and_places():
    import torch
    B, H, N, d = 1, 2, 8, 32
    Q, K, V = torch.zeros(B, 2 * H, N, d), torch.zeros(B, 2 * H, N, d), torch.zeros(B, H, N, 2 * d)
    lam, lens = torch.zeros(H), torch.zeros(B, dtype=torch.int32)
    O = torch.zeros(B, H, N, 2 * d)
    lse = torch.zeros(B, 2 * H, N)
    bad = [lambda: fbd.attn_diff_fwd(Q, K, V, lam),                     # on the CPU
           lambda: fbd.attn_diff_fwd(Q[:, :3], K, V, lam),              # an odd number of maps
           lambda: fbd.attn_diff_fwd(Q, K[:, :, :4], V, lam),           # another length
           lambda: fbd.attn_diff_fwd(Q, K, V[..., :d], lam),            # a value head of a map's width
           lambda: fbd.attn_diff_fwd(Q, K, V.bfloat16(), lam),
           lambda: fbd.attn_diff_fwd(Q, K, V, lam.double()),
           lambda: fbd.attn_diff_fwd(Q, K, V, lam[:1]),
           lambda: fbd.attn_diff_fwd(Q, K, V, lam, O=O[:, :1]),
           lambda: fbd.attn_diff_fwd(Q.half(), K.half(), V.half(), lam),
           lambda: fbd.attn_diff_fwd(Q, K, V, lam, bounds=(lens, lens)),
           lambda: fbd.attn_diff_bwd(Q, K, V, lam, O, O, O[:, :, :3], lse),
           lambda: fbd.attn_diff_bwd(Q, K, V, lam, O, O, O, lse[:, :1]),
           lambda: fbd.attn_diff_bwd(Q, K, V, lam, O, O, O, lse),       # on the CPU
           lambda: fbd.attn_diff_decode(Q, K, V, lam, lens),            # more than one token
           lambda: fbd.attn_diff_decode(Q[:, :, :1], K, V, lam, lens.long()),
           lambda: fbd.attn_diff_decode(Q[:, :, :1].contiguous(), K, V, lam, lens)]  # on the CPU
    pos, freq, axis = torch.zeros(3, N, dtype=torch.int32), torch.zeros(d // 2), torch.zeros(d // 2, dtype=torch.int32)
    bad += [lambda: fbd.attn_rope(Q, pos, freq, axis),                  # on the CPU
            lambda: fbd.attn_rope([Q] * 5, pos, freq, axis), lambda: fbd.attn_rope([], pos, freq, axis),
            lambda: fbd.attn_rope(Q, pos.long(), freq, axis), lambda: fbd.attn_rope(Q, pos[:, :3], freq, axis),
            lambda: fbd.attn_rope(Q, pos, freq[:3], axis), lambda: fbd.attn_rope(Q, pos, freq, axis.long()),
            lambda: fbd.attn_rope(Q, pos, freq, axis, paired="other"), lambda: fbd.attn_rope(Q[0], pos, freq, axis),
            lambda: fbd.attn_rope(Q, pos, freq, axis, outs=[Q, Q]),
            lambda: fbd.attn_rope(Q.transpose(2, 3), torch.zeros(3, d, dtype=torch.int32), freq[:4], axis[:4]),
            lambda: fbd.attn_rope((Q, V), pos, freq, axis)]
    for k, f in enumerate(bad):
        with pytest.raises(FbdError):
            f()
            raise AssertionError(f"case {k} was accepted")


@pytest.mark.parametrize("stream", [0, 1 << 40])
def test_refuses_host_tensors_given_a_stream(stream):
    import torch
    Q, V, lam = torch.zeros(1, 4, 8, 64), torch.zeros(1, 2, 8, 128), torch.zeros(2)
    with pytest.raises(FbdError):
        fbd.attn_diff_fwd(Q, Q, V, lam, stream=stream)
    with pytest.raises(FbdError):
        fbd.attn_rope([], torch.zeros(1, 8, dtype=torch.int32), lam, lam, stream=stream)
