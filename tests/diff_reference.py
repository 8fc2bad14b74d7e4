"""Plain 64-bit differential attention and rotary positions with torch, and for every output
the elementwise bound on what rounding may do to it: the tolerances of the parity tests.

u is half a step of the type the kernels round their operands to before a product (P, dS:
bf16 2^-8; float32: none), h half a step of the outputs' type.  FP32 (1e-5) covers the
exponentials' arguments (|s q.k| log2 e below 2^6 in units of 2^-24, and the approximate
2^x itself) and the fp32 sums, relative to the sum of the terms' magnitudes."""
from __future__ import annotations

import math

import torch

FP32 = 1e-5


def visible(N, mask, window=0, seg=None, device="cpu"):
    """[B or 1, N, N] truth values: row i sees key j."""
    i, j = torch.arange(N, device=device)[:, None], torch.arange(N, device=device)[None, :]
    v = torch.ones(N, N, dtype=torch.bool, device=device) if mask == "full" else j <= i
    if window:
        v = v & (j > i - window)
    v = v[None]
    if seg is not None:
        v = v & (seg[:, :, None] == seg[:, None, :])
    return v


def maps(Q, K, V, g):
    """Q [B, H, 2, N, d], K [B, H, 2, N, d], V [B, H, 1, N, 2d] in 64 bits, key/value heads repeated."""
    B, H2, N, d = Q.shape
    H = H2 // 2
    q = Q.double().view(B, H, 2, N, d)
    k = K.double().view(B, H // g, 2, K.shape[2], d).repeat_interleave(g, 1)
    v = V.double().unsqueeze(2).repeat_interleave(g, 1)
    return q, k, v


def forward(Q, K, V, lam, g, vis, scale=None):
    """O, O2, lse and the maps A [B, H, 2, N, N] (differentiable)."""
    q, k, v = maps(Q, K, V, g)
    s = scale or 1.0 / math.sqrt(q.shape[-1])
    S = (s * q @ k.transpose(-1, -2)).masked_fill(~vis[:, None, None], -math.inf)
    L = torch.logsumexp(S, -1)
    A = torch.exp(S - L[..., None])
    o = A @ v
    O = o[:, :, 0] - lam.double()[:, None, None] * o[:, :, 1]
    return O, o[:, :, 1], L.reshape(Q.shape[:3]), A


def with_bounds(Q, K, V, lam, dO, g, vis, scale=None):
    """{name: (value, bound)} of every output of the forward and the backward."""
    bf16 = Q.dtype == torch.bfloat16
    u, h = (2.0 ** -8, 2.0 ** -8) if bf16 else (0.0, 2.0 ** -24)
    B, H2, N, d = Q.shape
    H = H2 // 2
    s = scale or 1.0 / math.sqrt(d)
    q, k, v = maps(Q, K, V, g)
    O, O2, L, A = forward(Q, K, V, lam, g, vis, scale)
    la = lam.double().abs()[:, None, None]
    l1 = lam.double()[:, None, None]
    e = u + FP32
    mag = A @ v.abs()
    tO, tO2 = e * (mag[:, :, 0] + la * mag[:, :, 1]) + h * O.abs(), e * mag[:, :, 1] + h * O2.abs()
    out = {"O": (O, tO), "O2": (O2, tO2), "lse": (L, FP32 * (1 + L.abs()))}
    g_ = dO.double()
    dP = g_ @ v[:, :, 0].transpose(-1, -2)
    dPmag = g_.abs() @ v[:, :, 0].abs().transpose(-1, -2)
    D = (A * dP[:, :, None]).sum(-1)                                        # [B, H, 2, N]
    tD2 = (g_.abs() * (tO2 + FP32 * O2.abs())).sum(-1)
    tD1 = (g_.abs() * (tO + la * tO2 + FP32 * (O.abs() + la * O2.abs()))).sum(-1)
    w = torch.stack([torch.ones_like(l1), -l1], 2).view(1, H, 2, 1, 1)
    dS = w * A * (dP[:, :, None] - D[..., None])
    tS = e * dS.abs() + w.abs() * A * (torch.stack([tD1, tD2], 2)[..., None] + 1e-6 * dPmag[:, :, None])
    one = (vis.sum(-1) == 1)[:, None, None, :, None]                       # rows with one key: exactly zero
    dS, tS = dS.masked_fill(one, 0.0), tS.masked_fill(one, 0.0)
    dQ, tQ = s * dS @ k, s * tS @ k.abs()
    dK, tK = s * dS.transpose(-1, -2) @ q, s * tS.transpose(-1, -2) @ q.abs()
    W, tW = (w * A).sum(2), e * (w.abs() * A).sum(2)
    dV, tV = W.transpose(-1, -2) @ g_, tW.transpose(-1, -2) @ g_.abs()

    def shared(x):  # sums over the query heads of a key/value head
        return x.view(B, H // g, g, *x.shape[2:]).sum(2)

    dK, tK, dV, tV = shared(dK), shared(tK), shared(dV), shared(tV)
    out["dQ"] = (dQ.reshape(Q.shape), (tQ + h * dQ.abs()).reshape(Q.shape))
    out["dK"] = (dK.reshape(K.shape), (tK + h * dK.abs()).reshape(K.shape))
    out["dV"] = (dV, tV + h * dV.abs())
    out["dlam"] = (-D[:, :, 1].sum((0, 2)), (A[:, :, 1] * (FP32 * dP.abs() + 1e-6 * dPmag)).sum((0, 2, 3)) + 1e-30)
    return out


def rope(x, pos, freq, axis, paired="half", inverse=False):
    """The rotary of [B, heads, N, d] in 64 bits; pos [axes, B, N]."""
    x = x.double()
    d = x.shape[-1]
    turned = (axis >= 0) & (axis < pos.shape[0])
    p = pos.double()[axis.long().clamp(0, pos.shape[0] - 1)]                # [pairs, B, N]
    a = (p * freq.double()[:, None, None] * turned[:, None, None]).permute(1, 2, 0)[:, None]
    c, s = torch.cos(a), torch.sin(a) * (-1.0 if inverse else 1.0)
    u, v = (x[..., :d // 2], x[..., d // 2:]) if paired == "half" else (x[..., 0::2], x[..., 1::2])
    y, z = u * c - v * s, u * s + v * c
    return torch.cat([y, z], -1) if paired == "half" else torch.stack([y, z], -1).flatten(-2)
