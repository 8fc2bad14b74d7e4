"""Python binding of libfbd: exact attention (causal by default) forward, backward (GProj) and
backward-over-backward on GB300; differential attention (forward, backward, one token over a
cache) and multi-axis rotary positions; normed heads, a paged cache and the attention over it.

Argument marshalling only.  Every computation runs in the CUDA kernels of
``libfbd.so`` behind the C ABI declared in ``include/fbd.h``; PyTorch is used for
device memory and streams.  Importing the package loads the library and raises
if it is missing: there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import functools
import os

from . import _lib
from ._lib import (ATTN_BF16, ATTN_COL_PASS, ATTN_F32, ATTN_ROPE_HALF, ATTN_ROPE_MAX_TENSORS,  # noqa: F401
                   ATTN_ROPE_NEIGHBOUR, ATTN_ROW_PASS, AttnDesc, Cache, FbdError, NewTokens, NormGrad, NormTensor, RopeDesc,
                   RopeTensor, lib, status_name)

__all__ = [
    "attn_fwd", "attn_bwd", "attn_bob", "attn_bwd_passes", "attn_bob_passes", "ATTN_ROW_PASS", "ATTN_COL_PASS", "attn_bwd_workspace_bytes", "attn_bob_workspace_bytes",
    "attn_bob_static", "attn_bwd_projected_dS", "attn_segment_bounds",
    "attn_diff_fwd", "attn_diff_bwd", "attn_diff_bwd_workspace_bytes", "attn_diff_decode",
    "attn_diff_decode_workspace_bytes", "attn_rope", "attn_qk_norm", "attn_qk_norm_bwd", "attn_cache_append",
    "attn_paged", "attn_paged_workspace_bytes", "attn_device_status", "attn_check_wait_timeout",
    "attn_status_string", "attn_version", "make_desc",
    "FbdError", "AttnDesc", "ATTN_F32", "ATTN_BF16", "lib",
]

LIB_PATH = _lib.LIB_PATH


def _torch():
    import torch
    return torch


def _dtype_code(t) -> int:
    torch = _torch()
    if t.dtype == torch.float32:
        return ATTN_F32
    if t.dtype == torch.bfloat16:
        return ATTN_BF16
    raise FbdError(2, f"unsupported tensor dtype {t.dtype} (float32 or bfloat16)")


def make_desc(Q, scale: float = 0.0, causal: int = 1, K=None, window: int = 0, bounds=None) -> AttnDesc:
    """Descriptor from a [B, H, N, d] query tensor and, for grouped key/value heads,
    the [B, H / g, N, d] key tensor (g query heads per key/value head); window W > 0
    (with causal) limits query i to the keys i - W < j <= i; bounds = (seg_lo, seg_hi)
    from attn_segment_bounds sets the document mask (the descriptor keeps their device
    addresses: keep the tensors alive while it is used)."""
    if Q.dim() != 4 or (K is not None and K.dim() != 4):
        raise FbdError(1, "tensors must be [B, H, N, d]")
    B, H, N, d = Q.shape
    Hkv = H if K is None else K.shape[1]
    if (Hkv == 0) != (H == 0) or (Hkv and H % Hkv):
        raise FbdError(1, f"key/value heads ({Hkv}) must divide query heads ({H})")
    lo, hi = (None, None) if bounds is None else (_ptr(bounds[0]), _ptr(bounds[1]))
    return AttnDesc(B, H, N, d, float(scale), int(causal), _dtype_code(Q), H // Hkv if Hkv else 1, int(window),
                    lo, hi)


def _ptr(t):
    if t is None:
        return None
    if not t.is_contiguous():
        raise FbdError(1, "tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    torch = _torch()
    if stream is None:
        if torch.cuda.is_available():
            stream = torch.cuda.current_stream()
        else:
            return None
    return ctypes.c_void_p(int(getattr(stream, "cuda_stream", stream)))


def _check(status: int):
    if status != 0:
        raise FbdError(status, lib.attn_last_error().decode())


def attn_fwd(Q, K, V, O=None, lse=None, scale: float = 0.0, stream=None, desc=None, causal: bool = True, window: int = 0,
             bounds=None):
    """O, lse = attention forward (allocates O and lse with torch when not given)."""
    torch = _torch()
    desc = desc or make_desc(Q, scale, int(causal), K, window, bounds)
    if O is None:
        O = torch.empty_like(Q)
    if lse is None:
        lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device)
    _check(lib.attn_fwd(ctypes.byref(desc), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(lse), _stream(stream)))
    return O, lse


def attn_bwd_workspace_bytes(desc: AttnDesc, gproj: int = 0) -> int:
    return int(lib.attn_bwd_workspace_bytes(ctypes.byref(desc), int(gproj)))


def attn_bob_workspace_bytes(desc: AttnDesc, gproj: int = 0) -> int:
    return int(lib.attn_bob_workspace_bytes(ctypes.byref(desc), int(gproj)))


def _workspace(nbytes, like, workspace):
    torch = _torch()
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=like.device)
    return workspace


def attn_bwd(Q, K, V, O, dO, lse, gproj: int = 0, dQ=None, dK=None, dV=None, workspace=None,
             scale: float = 0.0, stream=None, desc=None, causal: bool = True, window: int = 0, bounds=None):
    """dQ, dK, dV = recompute backward (GProj when gproj != 0, bf16 only)."""
    return attn_bwd_passes(Q, K, V, O, dO, lse, ATTN_ROW_PASS | ATTN_COL_PASS, gproj, dQ, dK, dV, workspace,
                           scale, stream, desc, causal, window, bounds)


def attn_bwd_passes(Q, K, V, O, dO, lse, passes, gproj: int = 0, dQ=None, dK=None, dV=None, workspace=None,
                    scale: float = 0.0, stream=None, desc=None, causal: bool = True, window: int = 0, bounds=None):
    """The backward's row pass (dQ) and/or column pass (dK, dV); see attn_bwd_passes in fbd.h."""
    torch = _torch()
    desc = desc or make_desc(Q, scale, int(causal), K, window, bounds)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    need = attn_bwd_workspace_bytes(desc, gproj)
    workspace = _workspace(need, Q, workspace)
    _check(lib.attn_bwd_passes(ctypes.byref(desc), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(lse),
                               _ptr(dQ), _ptr(dK), _ptr(dV), int(gproj), _ptr(workspace),
                               ctypes.c_size_t(workspace.numel() * workspace.element_size()), int(passes),
                               _stream(stream)))
    return dQ, dK, dV


def attn_bob(Q, K, V, O, dO, lse, gdQ, gdK, gdV, gQ=None, gK=None, gV=None, gdO=None, workspace=None,
             scale: float = 0.0, stream=None, desc=None, causal: bool = True, window: int = 0, gproj: int = 0,
             bounds=None):
    """gQ, gK, gV, gdO = backward over backward against cotangents (gdQ, gdK, gdV)
    (GProj on the rounded dS of its dS b and dS^T a products when gproj != 0, bf16 only)."""
    return attn_bob_passes(Q, K, V, O, dO, lse, gdQ, gdK, gdV, ATTN_ROW_PASS | ATTN_COL_PASS, gQ, gK, gV, gdO,
                           workspace, scale, stream, desc, causal, window, gproj, bounds)


def attn_bob_passes(Q, K, V, O, dO, lse, gdQ, gdK, gdV, passes, gQ=None, gK=None, gV=None, gdO=None,
                    workspace=None, scale: float = 0.0, stream=None, desc=None, causal: bool = True, window: int = 0,
                    gproj: int = 0, bounds=None):
    """BoB's row pass (gQ, gdO, row states) and/or column pass (gK, gV); see fbd.h."""
    torch = _torch()
    desc = desc or make_desc(Q, scale, int(causal), K, window, bounds)
    gQ = torch.empty_like(Q) if gQ is None else gQ
    gK = torch.empty_like(K) if gK is None else gK
    gV = torch.empty_like(V) if gV is None else gV
    gdO = torch.empty_like(dO) if gdO is None else gdO
    workspace = _workspace(attn_bob_workspace_bytes(desc, gproj), Q, workspace)
    _check(lib.attn_bob_passes(ctypes.byref(desc), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(lse),
                               _ptr(gdQ), _ptr(gdK), _ptr(gdV), _ptr(gQ), _ptr(gK), _ptr(gV), _ptr(gdO), int(gproj),
                               _ptr(workspace), ctypes.c_size_t(workspace.numel() * workspace.element_size()),
                               int(passes), _stream(stream)))
    return gQ, gK, gV, gdO


def attn_bob_static(Q, K, V, O, dO, lse, gdQ, gdK, gdV, gQ=None, gK=None, gV=None, gdO=None,
                    scale: float = 0.0, stream=None, desc=None, causal: bool = True, window: int = 0, bounds=None):
    """attn_bob without a workspace argument: the library's static scratch array is used
    (for callers that cannot allocate device memory; B*H*Np <= 1,048,576 with Np = N
    rounded up to an even count)."""
    torch = _torch()
    desc = desc or make_desc(Q, scale, int(causal), K, window, bounds)
    gQ = torch.empty_like(Q) if gQ is None else gQ
    gK = torch.empty_like(K) if gK is None else gK
    gV = torch.empty_like(V) if gV is None else gV
    gdO = torch.empty_like(dO) if gdO is None else gdO
    _check(lib.attn_bob_static(ctypes.byref(desc), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(lse),
                               _ptr(gdQ), _ptr(gdK), _ptr(gdV), _ptr(gQ), _ptr(gK), _ptr(gV), _ptr(gdO),
                               _stream(stream)))
    return gQ, gK, gV, gdO


def attn_bwd_projected_dS(Q, K, V, O, dO, lse, dS=None, scale: float = 0.0, stream=None, desc=None, causal: bool = True,
                          window: int = 0, bounds=None):
    """Diagnostic: the GProj-projected dS [B, H, N, N] float32 (small N only)."""
    torch = _torch()
    desc = desc or make_desc(Q, scale, int(causal), K, window, bounds)
    B, H, N, _ = Q.shape
    dS = torch.empty((B, H, N, N), dtype=torch.float32, device=Q.device) if dS is None else dS
    _check(lib.attn_bwd_projected_dS(ctypes.byref(desc), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO),
                                     _ptr(lse), _ptr(dS), _stream(stream)))
    return dS


def attn_segment_bounds(seg, seg_lo=None, seg_hi=None, stream=None):
    """(seg_lo, seg_hi) int32 [B, N] of the document mask from segment ids seg [B, N]
    (int32, non-decreasing along N); pass them as `bounds` to the attention calls."""
    torch = _torch()
    if seg.dim() != 2 or seg.dtype != torch.int32:
        raise FbdError(1, "seg must be an int32 [B, N] tensor")
    B, N = seg.shape
    seg_lo = torch.empty_like(seg) if seg_lo is None else seg_lo
    seg_hi = torch.empty_like(seg) if seg_hi is None else seg_hi
    _check(lib.attn_segment_bounds(int(B), int(N), _ptr(seg), _ptr(seg_lo), _ptr(seg_hi), _stream(stream)))
    return seg_lo, seg_hi


def _on_stream(call):
    """A call given a stream runs under it as torch's current stream, so that what it allocates, the workspace above
    all, belongs to that stream and is not handed out again while the kernels there still use it."""

    @functools.wraps(call)
    def wrapped(*args, stream=None, **kwargs):
        if stream is None:
            return call(*args, **kwargs)
        torch, cuda = _torch(), _torch().cuda
        given = (t for v in (*args, *kwargs.values()) for t in (v if isinstance(v, (list, tuple)) else (v,)))
        device = next((t.device for t in given if torch.is_tensor(t) and t.is_cuda), None)
        if device is None:  # refused there, or nothing to launch
            return call(*args, **kwargs)
        if isinstance(stream, cuda.Stream):
            if stream.device != device:
                raise FbdError(1, f"a stream of {stream.device} for tensors on {device}")
        else:  # a handle: a stream of the tensors' device, 0 (and cudaStreamLegacy, 1) its default one
            handle = int(getattr(stream, "cuda_stream", stream))
            stream = cuda.ExternalStream(handle, device=device) if handle > 1 else cuda.default_stream(device)
        with cuda.stream(stream):
            return call(*args, **kwargs)

    return wrapped


def _launch(fn, tensors, *args):
    """fn(*args, stream) on the device the tensors are on: one CUDA device, made current for the call, and its current
    stream.  Empty tensors launch nothing, so they may be anywhere."""
    cuda = _torch().cuda
    devices = {t.get_device() for t in tensors if t is not None}
    if len(devices) > 1 or -1 in devices:
        devices = {t.get_device() for t in tensors if t is not None and t.numel()}
    if len(devices) > 1 or -1 in devices:
        raise FbdError(1, f"tensors must be on one CUDA device (got {sorted({str(t.device) for t in tensors if t is not None})})")
    if not devices:
        _check(fn(*args, None))
        return
    device = devices.pop()
    stream = cuda.current_stream(device).cuda_stream
    if device == cuda.current_device():
        _check(fn(*args, stream))
    else:
        with cuda.device(device):
            _check(fn(*args, stream))


def _at(name, t):
    """Address of a contiguous tensor."""
    if not t.is_contiguous():
        raise FbdError(1, f"{name} must be contiguous")
    return t.data_ptr()


def _want(name, t, shape, dtype):
    """The address of t, contiguous and of that shape and type."""
    if t is None:
        raise FbdError(1, f"{name} is None")
    if t.shape != shape or t.dtype != dtype:
        raise FbdError(1, f"{name} must be {dtype} {tuple(shape)} (got {t.dtype} {tuple(t.shape)})")
    return _at(name, t)


def _diff_desc(Q, K, V, lam, scale, causal, window, bounds, queries=None):
    """Descriptor of a differential attention call (queries: 1 for a token over a cache, None where Q has the keys'
    length) and the addresses of Q, K, V and lam, their shapes and types checked."""
    if any(t is None or t.dim() != 4 for t in (Q, K, V)):
        raise FbdError(1, "Q, K and V must be 4-dimensional tensors")
    dtype = Q.dtype
    B, maps, _, d = Q.shape
    _, kmaps, N, _ = K.shape
    if maps % 2 or kmaps % 2:
        raise FbdError(1, f"Q and K hold two maps per head, got {maps} and {kmaps} slices")
    H, Hkv = maps // 2, kmaps // 2
    if (Hkv == 0) != (H == 0) or (Hkv and H % Hkv):
        raise FbdError(1, f"key/value heads ({Hkv}) must divide query heads ({H})")
    ptrs = (_want("Q", Q, (B, maps, N if queries is None else queries, d), dtype), _want("K", K, (B, kmaps, N, d), dtype),
            _want("V", V, (B, Hkv, N, 2 * d), dtype), _want("lam", lam, (H,), _torch().float32))
    lo = hi = None
    if bounds is not None:
        lo, hi = (_want(name, t, (B, N), _torch().int32) for name, t in zip(("seg_lo", "seg_hi"), bounds))
    window = max(-1, min(window, max(N, 1)))  # (the field has 32 bits; N or more is no window)
    return AttnDesc(B, H, N, d, scale, causal, _dtype_code(Q), H // Hkv if Hkv else 1, window, lo, hi), ptrs


@_on_stream
def attn_diff_fwd(Q, K, V, lam, O=None, O2=None, lse=None, scale: float = 0.0, causal: bool = True, window: int = 0,
                  bounds=None, for_backward: bool = True):
    """O, O2, lse = differential attention (A_1 - lam_h A_2) V of Q [B, 2H, N, d], K [B, 2H/g, N, d] (the maps of a
    head in neighbouring slices), V [B, H/g, N, 2d], lam [H] float32.  O2 = A_2 V and lse are what the backward
    needs; for_backward=False leaves O2 out (returned as None).  stream=: the stream to run on (keyword only)."""
    torch = _torch()
    desc, ptrs = _diff_desc(Q, K, V, lam, scale, causal, window, bounds)
    shape = (desc.B, desc.H, desc.N, 2 * desc.d)
    if O is None:
        O = torch.empty(shape, dtype=Q.dtype, device=Q.device)
    if O2 is None and for_backward:
        O2 = torch.empty_like(O)
    if lse is None:
        lse = torch.empty(Q.shape[:3], dtype=torch.float32, device=Q.device)
    outs = (_want("O", O, shape, Q.dtype), None if O2 is None else _want("O2", O2, shape, Q.dtype),
            _want("lse", lse, Q.shape[:3], torch.float32))
    _launch(lib.attn_diff_fwd, (Q, K, V, lam, O, O2, lse, *(bounds or ())), ctypes.byref(desc), *ptrs, *outs)
    return O, O2, lse


def attn_diff_bwd_workspace_bytes(desc: AttnDesc) -> int:
    return int(lib.attn_diff_bwd_workspace_bytes(ctypes.byref(desc)))


@_on_stream
def attn_diff_bwd(Q, K, V, lam, O, O2, dO, lse, dQ=None, dK=None, dV=None, dlam=None, workspace=None,
                  scale: float = 0.0, causal: bool = True, window: int = 0, bounds=None):
    """dQ, dK, dV, dlam = recompute backward of attn_diff_fwd (its mask and scale given again)."""
    torch = _torch()
    desc, ptrs = _diff_desc(Q, K, V, lam, scale, causal, window, bounds)
    shape, dtype = (desc.B, desc.H, desc.N, 2 * desc.d), Q.dtype
    ins = (_want("O", O, shape, dtype), _want("O2", O2, shape, dtype), _want("dO", dO, shape, dtype),
           _want("lse", lse, Q.shape[:3], torch.float32))
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    dlam = torch.empty_like(lam) if dlam is None else dlam
    outs = (_want("dQ", dQ, Q.shape, dtype), _want("dK", dK, K.shape, dtype), _want("dV", dV, V.shape, dtype),
            _want("dlam", dlam, lam.shape, torch.float32))
    workspace = _workspace(lib.attn_diff_bwd_workspace_bytes(ctypes.byref(desc)), Q, workspace)
    _launch(lib.attn_diff_bwd, (Q, K, V, lam, O, O2, dO, lse, dQ, dK, dV, dlam, workspace if Q.numel() else None,
                                *(bounds or ())), ctypes.byref(desc), *ptrs, *ins, *outs, _at("workspace", workspace),
            workspace.nbytes)
    return dQ, dK, dV, dlam


def attn_diff_decode_workspace_bytes(desc: AttnDesc) -> int:
    return int(lib.attn_diff_decode_workspace_bytes(ctypes.byref(desc)))


@_on_stream
def attn_diff_decode(Q, K, V, lam, lens, O=None, workspace=None, scale: float = 0.0, window: int = 0):
    """O [B, H, 1, 2d] = differential attention of one token per sequence, Q [B, 2H, 1, d], over a cache K
    [B, 2H/g, capacity, d], V [B, H/g, capacity, 2d] of which sequence b holds lens[b] keys (int32, on the device;
    the new token's among them).  A sequence without a key gives zeros."""
    torch = _torch()
    desc, ptrs = _diff_desc(Q, K, V, lam, scale, True, window, None, queries=1)
    shape = (desc.B, desc.H, 1, 2 * desc.d)
    lens_at = _want("lens", lens, (desc.B,), torch.int32)
    if O is None:
        O = torch.empty(shape, dtype=Q.dtype, device=Q.device)
    O_at = _want("O", O, shape, Q.dtype)
    workspace = _workspace(lib.attn_diff_decode_workspace_bytes(ctypes.byref(desc)), Q, workspace)
    _launch(lib.attn_diff_decode, (Q, K, V, lam, lens, O, workspace if Q.numel() else None), ctypes.byref(desc), *ptrs,
            lens_at, O_at, _at("workspace", workspace), workspace.nbytes)
    return O


@_on_stream
def attn_rope(xs, pos, freq, axis, outs=None, paired: str = "half", inverse: bool = False):
    """Rotary positions with several axes: pair i of each token of the [B, heads, N, d] views `xs` (one tensor or up to
    four, any strides with d contiguous) turns by freq[i] * pos[axis[i]]; pos [axes, B, N] or [axes, N] int32, freq
    [d/2] float32, axis [d/2] int32 (-1: the pair is copied unturned).  paired: "half" (coordinates i, i + d/2) or
    "neighbour" (2i, 2i + 1).  inverse=True turns back (the gradient).  Returns `outs` (contiguous [B, heads, N, d]
    tensors when not given; views of any strides when given, x itself among them), one tensor for one."""
    torch = _torch()
    single = torch.is_tensor(xs)
    xs = [xs] if single else list(xs or ())
    if not 1 <= len(xs) <= ATTN_ROPE_MAX_TENSORS:
        raise FbdError(1, f"1 to {ATTN_ROPE_MAX_TENSORS} tensors, got {len(xs)}")
    if any(x is None or x.dim() != 4 for x in xs):
        raise FbdError(1, "tensors must be [B, heads, N, d]")
    if outs is None:
        outs = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in xs]
    else:
        outs = [outs] if torch.is_tensor(outs) else list(outs)
    if len(outs) != len(xs):
        raise FbdError(1, f"{len(xs)} inputs and {len(outs)} outputs")
    if paired not in ("half", "neighbour"):
        raise FbdError(1, f"paired must be 'half' or 'neighbour' (got {paired!r})")
    B, _, N, d = xs[0].shape
    dtype = xs[0].dtype
    tensors = (RopeTensor * len(xs))()
    for t, x, y in zip(tensors, xs, outs):
        heads = x.shape[1]
        if x.shape != (B, heads, N, d) or y.shape != x.shape or x.dtype != dtype or y.dtype != dtype:
            raise FbdError(1, f"tensors must be {dtype} [{B}, heads, {N}, {d}], an output like its input (got "
                              f"{x.dtype} {tuple(x.shape)} and {y.dtype} {tuple(y.shape)})")
        xs_, ys_ = x.stride(), y.stride()
        if heads and B and N and (xs_[3] != 1 or ys_[3] != 1):
            raise FbdError(1, "the last dimension must be contiguous")
        t.x, t.y, t.heads, t.x_stride[:], t.y_stride[:] = x.data_ptr(), y.data_ptr(), heads, xs_[:3], ys_[:3]
    if pos is None or pos.dim() not in (2, 3):
        raise FbdError(1, "pos must be [axes, B, N] or [axes, N]")
    axes, shared = pos.shape[0], pos.dim() == 2
    tables = (_want("pos", pos, (axes, N) if shared else (axes, B, N), torch.int32),
              _want("freq", freq, (d // 2,), torch.float32), _want("axis", axis, (d // 2,), torch.int32))
    desc = RopeDesc(B, N, d, axes, _dtype_code(xs[0]), ATTN_ROPE_HALF if paired == "half" else ATTN_ROPE_NEIGHBOUR,
                    bool(inverse), 0 if shared else N)
    _launch(lib.attn_rope, (*xs, *outs, pos, freq, axis) if any(x.numel() for x in xs) else (),
            ctypes.byref(desc), tensors, len(xs), *tables)
    return outs[0] if single else outs


def _view(name, x, shape, dtype, strides):
    """The address of a view [B, heads, N, d] of that shape and type, its last dimension contiguous; its strides of the
    other three into `strides`."""
    if x is None:
        raise FbdError(1, f"{name} is None")
    if x.shape != shape or x.dtype != dtype:
        raise FbdError(1, f"{name} must be {dtype} {tuple(shape)} (got {x.dtype} {tuple(x.shape)})")
    strides[0], strides[1], strides[2], last = x.stride()
    if last != 1 and x.numel():
        raise FbdError(1, f"the last dimension of {name} must be contiguous")
    return x.data_ptr()


def _angles(pos, freq, axis, B, N, d, own_pos=False):
    """(axes, shared, addresses of pos, freq, axis) of a rotary's tables, all None where nothing turns; own_pos: pos may
    be left out alone (the tokens' own positions)."""
    torch = _torch()
    if pos is None and freq is None and axis is None:
        return 1, True, (None, None, None)
    at = None
    axes, shared = 1, True
    if pos is not None or not own_pos:
        if pos is None or pos.dim() not in (2, 3):
            raise FbdError(1, "pos must be [axes, B, N] or [axes, N]")
        axes, shared = pos.shape[0], pos.dim() == 2
        at = _want("pos", pos, (axes, N) if shared else (axes, B, N), torch.int32)
    return axes, shared, (at, _want("freq", freq, (d // 2,), torch.float32), _want("axis", axis, (d // 2,), torch.int32))


def _norm_desc(xs, pos, freq, axis, paired):
    """Descriptor of a call on normed heads, the shape [B, heads, N, d] of its first tensor, and its tables."""
    if not 1 <= len(xs) <= ATTN_ROPE_MAX_TENSORS:
        raise FbdError(1, f"1 to {ATTN_ROPE_MAX_TENSORS} tensors, got {len(xs)}")
    for x in xs:
        if x is None or x.dim() != 4:
            raise FbdError(1, "tensors must be [B, heads, N, d]")
    if paired not in ("half", "neighbour"):
        raise FbdError(1, f"paired must be 'half' or 'neighbour' (got {paired!r})")
    B, _, N, d = xs[0].shape
    axes, shared, tables = _angles(pos, freq, axis, B, N, d)
    desc = RopeDesc(B, N, d, axes, _dtype_code(xs[0]), ATTN_ROPE_HALF if paired == "half" else ATTN_ROPE_NEIGHBOUR, 0,
                    0 if shared else N)
    return desc, (B, N, d), tables


def _listed(ts, n, what):
    """A tensor, None or a list of n of them as a list."""
    if ts is None:
        return [None] * n
    ts = list(ts) if isinstance(ts, (list, tuple)) or not _torch().is_tensor(ts) else [ts]
    if len(ts) != n:
        raise FbdError(1, f"{n} tensors and {len(ts)} {what}")
    return ts


@_on_stream
def attn_qk_norm(xs, weights=None, pos=None, freq=None, axis=None, outs=None, paired: str = "half", eps: float = 1e-6):
    """RMS norm over d of each head's vector, z = w x / sqrt(mean x^2 + eps), then the turn of attn_rope, in one pass over
    the [B, heads, N, d] views `xs` (one tensor or up to four, any strides with d contiguous).  weights: float32 [d] per
    tensor (None: ones).  pos, freq, axis: as in attn_rope, all None: no turn.  Returns `outs` (contiguous [B, heads, N, d]
    tensors when not given; views when given, x itself among them), one tensor for one."""
    torch = _torch()
    single = torch.is_tensor(xs)
    xs = [xs] if single else list(xs or ())
    desc, (B, N, d), tables = _norm_desc(xs, pos, freq, axis, paired)
    weights = _listed(weights, len(xs), "weights")
    outs = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in xs] if outs is None else _listed(outs, len(xs), "outputs")
    tensors = (NormTensor * len(xs))()
    for t, x, w, y in zip(tensors, xs, weights, outs):
        shape = (B, x.shape[1], N, d)
        t.x, t.y = _view("x", x, shape, xs[0].dtype, t.x_stride), _view("an output", y, shape, xs[0].dtype, t.y_stride)
        t.w, t.heads = None if w is None else _want("weight", w, (d,), torch.float32), shape[1]
    _launch(lib.attn_qk_norm, (*xs, *outs, *weights, pos, freq, axis) if any(x.numel() for x in xs) else (),
            ctypes.byref(desc), tensors, len(xs), eps, *tables)
    return outs[0] if single else outs


@_on_stream
def attn_qk_norm_bwd(xs, dys, weights=None, pos=None, freq=None, axis=None, dxs=None, dweights=None, workspace=None,
                     paired: str = "half", eps: float = 1e-6):
    """dxs, dweights = gradient of attn_qk_norm at xs for the gradients dys of its outputs (the tables, weights and eps
    given again).  dxs: contiguous tensors when not given, x or dy itself among those given; dweights: float32 [d] per
    tensor, None where its weight is None.  One tensor each for one tensor."""
    torch = _torch()
    single = torch.is_tensor(xs)
    xs = [xs] if single else list(xs or ())
    desc, (B, N, d), tables = _norm_desc(xs, pos, freq, axis, paired)
    dys = _listed(dys, len(xs), "gradients")
    weights = _listed(weights, len(xs), "weights")
    dxs = [torch.empty(x.shape, dtype=x.dtype, device=x.device) for x in xs] if dxs is None else _listed(dxs, len(xs), "dxs")
    dweights = [None if w is None else torch.empty_like(w) for w in weights] if dweights is None else \
        _listed(dweights, len(xs), "dweights")
    tensors = (NormGrad * len(xs))()
    dtype = xs[0].dtype
    for t, x, dy, dx, w, dw in zip(tensors, xs, dys, dxs, weights, dweights):
        shape = (B, x.shape[1], N, d)
        t.x, t.dy, t.dx = (_view("x", x, shape, dtype, t.x_stride), _view("dy", dy, shape, dtype, t.dy_stride),
                           _view("dx", dx, shape, dtype, t.dx_stride))
        t.w = None if w is None else _want("weight", w, (d,), torch.float32)
        t.dw = None if dw is None else _want("dweight", dw, (d,), torch.float32)
        t.heads = shape[1]
    workspace = _workspace(lib.attn_qk_norm_bwd_workspace_bytes(ctypes.byref(desc), tensors, len(xs)), xs[0], workspace)
    some = any(x.numel() for x in xs)
    _launch(lib.attn_qk_norm_bwd, (*xs, *dys, *dxs, *weights, *dweights, pos, freq, axis, workspace) if some else dweights,
            ctypes.byref(desc), tensors, len(xs), eps, *tables, _at("workspace", workspace), workspace.nbytes)
    return (dxs[0], dweights[0]) if single else (dxs, dweights)


def _cache_of(cache, heads, d, dtype, B):
    """The C structure of a cache (K, V, table)."""
    try:
        K, V, table = cache
    except (TypeError, ValueError):
        raise FbdError(1, "a cache is (K, V, table)") from None
    if K is None or V is None or table is None or K.dim() != 4:
        raise FbdError(1, "a cache is K and V [pages, heads, page_size, d] and table [B, width]")
    c = Cache()
    shape = (K.shape[0], heads, K.shape[2], d)
    c.K, c.V = _view("K of the cache", K, shape, dtype, c.k_stride), _view("V of the cache", V, shape, dtype, c.v_stride)
    c.table = _want("table", table, (B, table.shape[-1] if table.dim() else 0), _torch().int32)
    c.pages, c.page_size, c.width = K.shape[0], K.shape[2], table.shape[1]
    return c, (K, V, table)


def _sequences(lens, cu, batch):
    """(B, addresses of cu and lens) of a call's sequences; batch: of its [batch, heads, N, d] tensors."""
    torch = _torch()
    if lens is None or lens.dim() != 1:
        raise FbdError(1, "lens must be an int32 [B] tensor")
    B = lens.shape[0]
    if batch != (B if cu is None else 1):
        raise FbdError(1, f"{batch} batch rows for {B} sequences" + ("" if cu is None else " of packed tokens (one batch row)"))
    return B, (None if cu is None else _want("cu", cu, (B + 1,), torch.int32), _want("lens", lens, (B,), torch.int32))


@_on_stream
def attn_cache_append(K, V, cache, lens, cu=None, Q=None, Q_out=None, weights=None, pos=None, freq=None, axis=None,
                      paired: str = "half", eps: float = 1e-6):
    """The new tokens' K and V [B, Hkv, N, d] into the pages of `cache` = (K, V [pages, Hkv, page_size, d], table [B, width]
    int32), the keys normed and turned on the way, and the queries Q [B, H, N, d] too if given.  lens [B] int32: the keys
    each sequence holds then; cu [B + 1] int32: packed tokens, views [1, heads, N, d] of which sequence b has the rows
    cu[b] .. cu[b + 1] - 1.  weights = (wq, wk), float32 [d] or None each: the norm of attn_qk_norm (None: no norm).
    freq, axis: attn_rope's tables (None: no turn), pos None: the tokens' positions in their sequences.  Returns Q_out
    (a contiguous tensor when not given, Q itself among those given; rows of no sequence stay as they were), None
    without Q."""
    torch = _torch()
    if any(x is None or x.dim() != 4 for x in (K, V)) or (Q is not None and Q.dim() != 4):
        raise FbdError(1, "tensors must be [B, heads, N, d]")
    if paired not in ("half", "neighbour"):
        raise FbdError(1, f"paired must be 'half' or 'neighbour' (got {paired!r})")
    dtype = K.dtype
    batch, Hkv, N, d = K.shape
    B, (cu_at, lens_at) = _sequences(lens, cu, batch)
    H = Hkv if Q is None else Q.shape[1]
    if (Hkv == 0) != (H == 0) or (Hkv and H % Hkv):
        raise FbdError(1, f"key/value heads ({Hkv}) must divide query heads ({H})")
    c, parts = _cache_of(cache, Hkv, d, dtype, B)
    t = NewTokens()
    t.K, t.V = _view("K", K, K.shape, dtype, t.k_stride), _view("V", V, K.shape, dtype, t.v_stride)
    if Q is None and Q_out is not None:
        raise FbdError(1, "Q_out without Q")
    if Q is not None:
        if Q_out is None:
            Q_out = torch.empty(Q.shape, dtype=dtype, device=Q.device)
        shape = (batch, H, N, d)
        t.Q, t.Q_out = _view("Q", Q, shape, dtype, t.q_stride), _view("Q_out", Q_out, shape, dtype, t.q_out_stride)
    wq, wk = (None, None) if weights is None else _listed(weights, 2, "weights")
    t.q_weight, t.k_weight = (None if w is None else _want("weight", w, (d,), torch.float32) for w in (wq, wk))
    axes, shared, (t.pos, t.freq, t.axis) = _angles(pos, freq, axis, batch, N, d, own_pos=True)
    t.pos_batch_stride, t.axes = 0 if shared else N, axes
    t.paired = ATTN_ROPE_HALF if paired == "half" else ATTN_ROPE_NEIGHBOUR
    t.normed, t.eps = weights is not None, eps
    desc = AttnDesc(B, H, N, d, 0.0, 1, _dtype_code(K), H // Hkv if Hkv else 1, 0, None, None)
    _launch(lib.attn_cache_append, (K, V, *parts, lens, cu, Q, Q_out, wq, wk, pos, freq, axis) if K.numel() else (),
            ctypes.byref(desc), ctypes.byref(t), ctypes.byref(c), cu_at, lens_at)
    return Q_out


def attn_paged_workspace_bytes(desc: AttnDesc, max_new: int = 0) -> int:
    return int(lib.attn_paged_workspace_bytes(ctypes.byref(desc), int(max_new)))


_Strides = ctypes.c_int64 * 3


@_on_stream
def attn_paged(Q, cache, lens, cu=None, O=None, lse=None, workspace=None, scale: float = 0.0, causal: bool = True,
               window: int = 0, max_new: int = 0):
    """O, lse = attention of the new tokens Q [B, H, N, d] over a paged cache = (K, V [pages, Hkv, page_size, d], table
    [B, width] int32) that holds lens [B] int32 keys of each sequence, the new tokens' own among them (they are its last
    ones).  cu [B + 1] int32: packed tokens, Q [1, H, N, d], sequence b has the rows cu[b] .. cu[b + 1] - 1.  Q, K, V and O
    are views of any strides with d contiguous; O is given its memory token by token ([B, N, H, d]) when it is not given,
    as a layer's output projection takes it.  lse float32 [B, H, N].  max_new: the most new tokens of a sequence, where the
    host knows it (1 when each has one): it chooses the kernel and may change roundings, nothing else, and a workspace given
    is sized with the same one (N without cu).  A token that sees no key gives O = 0, lse = -inf; rows of no sequence stay
    as they were."""
    torch = _torch()
    if Q is None or Q.dim() != 4:
        raise FbdError(1, "Q must be [B, H, N, d]")
    dtype = Q.dtype
    batch, H, N, d = Q.shape
    B, (cu_at, lens_at) = _sequences(lens, cu, batch)
    Hkv = cache[0].shape[1] if isinstance(cache, (tuple, list)) and len(cache) == 3 and getattr(cache[0], "ndim", 0) == 4 else 0
    if (Hkv == 0) != (H == 0) or (Hkv and H % Hkv):
        raise FbdError(1, f"key/value heads ({Hkv}) must divide query heads ({H})")
    c, parts = _cache_of(cache, Hkv, d, dtype, B)
    if O is None:
        O = torch.empty((batch, N, H, d), dtype=dtype, device=Q.device).transpose(1, 2)
    if lse is None:
        lse = torch.empty((batch, H, N), dtype=torch.float32, device=Q.device)
    qs, os_ = _Strides(), _Strides()
    Q_at, O_at = _view("Q", Q, Q.shape, dtype, qs), _view("O", O, Q.shape, dtype, os_)
    lse_at = _want("lse", lse, (batch, H, N), torch.float32)
    window = max(-1, min(window, (1 << 31) - 1))  # (the field has 32 bits; positions are below 2^31 - 1, so that much is no window)
    desc = AttnDesc(B, H, N, d, scale, causal, _dtype_code(Q), H // Hkv if Hkv else 1, window, None, None)
    max_new = N if cu is None else min(max_new, N)
    workspace = _workspace(lib.attn_paged_workspace_bytes(ctypes.byref(desc), max_new), Q, workspace)
    _launch(lib.attn_paged, (Q, *parts, lens, cu, O, lse, workspace) if Q.numel() and B else (), ctypes.byref(desc), Q_at, qs,
            ctypes.byref(c), cu_at, lens_at, max_new, O_at, os_, lse_at, _at("workspace", workspace), workspace.nbytes)
    return O, lse


def attn_device_status(stream=None) -> int:
    """Synchronise the stream; raise FbdError if a device-side wait timed out."""
    _check(lib.attn_device_status(_stream(stream)))
    return 0


def attn_check_wait_timeout(stream=None) -> int:
    """Run the library's failure-detection check (a bounded device wait that is made to
    give up); returns the status code, ATTN_ERR_TIMEOUT (6) when the path works."""
    return int(lib.attn_check_wait_timeout(_stream(stream)))


def attn_status_string(status: int) -> str:
    return lib.attn_status_string(int(status)).decode()


def attn_version() -> str:
    return lib.attn_version().decode()
