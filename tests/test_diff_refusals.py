"""Refusals of the differential attention and rotary entry points that need no GPU (fake pointers,
never dereferenced): rotary outputs over another tensor or over a table; an input left out."""
import ctypes

import pytest

import __graft_entry__

__graft_entry__.build()
import fwd_bwd_double_gb300 as fbd  # noqa: E402
from fwd_bwd_double_gb300 import RopeDesc, RopeTensor, lib  # noqa: E402

INVALID = 1
B, N, D, HEADS = 2, 8, 64, 4
BYTES = B * HEADS * N * D * 2
X0, Y0, X1, Y1, POS, FREQ, AXIS = ((1 << 40) + k * (1 << 32) for k in range(7))


def rope(x0=X0, y0=Y0, x1=X1, y1=Y1, pos=POS, freq=FREQ, axis=AXIS, xs=None):
    t = (RopeTensor * 2)()
    for k, (x, y) in enumerate(((x0, y0), (x1, y1))):
        t[k].x, t[k].y, t[k].heads = x, y, HEADS
        t[k].x_stride[:] = xs or (HEADS * N * D, N * D, D)
        t[k].y_stride[:] = (HEADS * N * D, N * D, D)
    desc = RopeDesc(B, N, D, 3, 1, 0, 0, N)
    return lib.attn_rope(ctypes.byref(desc), t, 2, *(ctypes.c_void_p(p) for p in (pos, freq, axis)), None)


@pytest.mark.parametrize("kw", [
    dict(y0=X1, y1=X0),                     # outputs and inputs crossed
    dict(y0=X1), dict(y1=X0), dict(y0=X0, y1=X0),
    dict(y1=Y0), dict(y1=Y0 + BYTES - 16), dict(y0=Y1 + BYTES - 16),
    dict(x1=X0, y0=X0),                     # the second tensor reads what the first writes in place
    dict(y0=X0 + 16), dict(y0=X1 + BYTES - 16), dict(y1=X0 - BYTES + 16),
    dict(pos=Y0), dict(pos=Y1 + BYTES - 4), dict(pos=Y1 - 3 * B * N * 4 + 4), dict(freq=Y0 + 64), dict(freq=Y1 - D * 2 + 4),
    dict(axis=Y1 + BYTES - 4), dict(axis=Y0),
    dict(xs=(0, 0, D), y0=X0 + 16), dict(xs=(0, 0, D), y1=X0),   # a broadcast input
])
def test_rope_refuses_outputs_over_other_tensors_and_tables(kw):
    assert rope(**kw) == INVALID
    assert b"overlaps" in lib.attn_last_error()


def test_binding_refuses_an_input_left_out():
    """None for a tensor, O2 above all, which a forward without the backward's output returns."""
    import torch
    Q, V, lam, lse = torch.zeros(1, 4, 8, 32), torch.zeros(1, 2, 8, 64), torch.zeros(2), torch.zeros(1, 4, 8)
    ins = (Q, Q, V, lam, V, V, V, lse)
    for k in range(len(ins)):
        with pytest.raises(fbd.FbdError):
            fbd.attn_diff_bwd(*(None if u == k else t for u, t in enumerate(ins)))
    for k in range(4):
        with pytest.raises(fbd.FbdError):
            fbd.attn_diff_fwd(*(None if u == k else t for u, t in enumerate(ins[:4])))
    token = (Q[:, :, :1].contiguous(), Q, V, lam, torch.zeros(1, dtype=torch.int32))
    for k in range(5):
        with pytest.raises(fbd.FbdError):
            fbd.attn_diff_decode(*(None if u == k else t for u, t in enumerate(token)))
    tables = (torch.zeros(1, 8, dtype=torch.int32), torch.zeros(16), torch.zeros(16, dtype=torch.int32))
    for k in range(4):
        with pytest.raises(fbd.FbdError):
            fbd.attn_rope(*(None if u == k else t for u, t in enumerate((Q, *tables))))
    with pytest.raises(fbd.FbdError):
        fbd.attn_rope((Q, None), *tables)


@pytest.mark.parametrize("window,taken", [(0, 0), (5, 5), (8, 8), (1 << 31, 8), ((1 << 32) + 5, 8), (1 << 70, 8), (-1, -1),
                                          (5 - (1 << 32), -1)])
def test_a_window_past_32_bits_is_none(window, taken):
    """The descriptor's window has 32 bits: one as wide as the sequence or wider is no window at all;
    a negative one stays negative, which is refused."""
    import torch
    Q, V, lam = torch.zeros(1, 4, 8, 32), torch.zeros(1, 2, 8, 64), torch.zeros(2)
    desc, _ = fbd._diff_desc(Q, Q, V, lam, 0.0, True, window, None)
    assert desc.window == taken
