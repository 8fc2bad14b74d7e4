"""Plain 64-bit normed heads, appends to a paged cache and attention over it, with torch, and for
every output the elementwise bound on what rounding may do to it: the tolerances of the parity tests.

u is half a step of the type the kernels round the probabilities to before their product (bf16 2^-8;
float32: none), h half a step of the outputs' type.  FP32 (1e-5) covers the exponentials' arguments
(|s q.k| log2 e below 2^6 in units of 2^-24, and the approximate 2^x itself) and the fp32 sums, relative
to the sum of the terms' magnitudes.  NORM (4e-6) covers a head's norm and turn: a sum of at most 256
squares in chains of 16 and 5 (21 roundings of 2^-24, halved by the square root), the reciprocal root
(2^-22), sine and cosine (2^-22), and some six products and sums (2^-24 each): below 2e-6, doubled.  ANGLE: an angle's own
rounding, which a sine near 0 or 1 passes on whole: in units of pi it is at most 1 in magnitude, so
its float32 is within 2^-25, pi 2^-25 = 9.4e-8 radians, and it is formed within 2^-32 of a turn (1.5e-9)."""
from __future__ import annotations

import math

import torch

FP32 = 1e-5
NORM = 4e-6
ANGLE = 1e-7


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def pairs(t, paired):
    d = t.shape[-1]
    return (t[..., :d // 2], t[..., d // 2:]) if paired == "half" else (t[..., 0::2], t[..., 1::2])


def joined(u, v, paired):
    return torch.cat([u, v], -1) if paired == "half" else torch.stack([u, v], -1).flatten(-2)


def cos_sin(pos, freq, axis):
    """[B, 1, N, pairs] in 64 bits of pos [axes, B, N]; axes outside 0 .. axes - 1 do not turn."""
    turned = (axis >= 0) & (axis < pos.shape[0])
    p = pos.double()[axis.long().clamp(0, pos.shape[0] - 1)]
    a = (p * freq.double()[:, None, None] * turned[:, None, None]).permute(1, 2, 0)[:, None]
    return torch.cos(a), torch.sin(a)


def turn(t, cs, paired, inverse=False):
    """t turned, and the sum of its terms' magnitudes, the angle's error among them in units of NORM."""
    if cs is None:
        return t, t.abs()
    c, s = cs
    s = -s if inverse else s
    u, v = pairs(t, paired)
    off = ANGLE / NORM * (u.abs() + v.abs())
    return (joined(u * c - v * s, u * s + v * c, paired),
            joined(u.abs() * c.abs() + v.abs() * s.abs() + off, u.abs() * s.abs() + v.abs() * c.abs() + off, paired))


def rms(x, eps):
    return (x.double().square().mean(-1, keepdim=True) + eps) ** -0.5


def norm(x, w, cs, paired="half", eps=1e-6):
    """y and its bound; w None: ones."""
    z = x.double() * rms(x, eps) * (1.0 if w is None else w.double())
    y, mag = turn(z, cs, paired)
    return y, NORM * mag + half_step(x.dtype) * y.abs() + 1e-37


def norm_bwd(x, w, dy, cs, paired="half", eps=1e-6):
    """(dx, bound), (dw, bound)."""
    r = rms(x, eps)
    dz, mz = turn(dy.double(), cs, paired, inverse=True)
    n = x.double() * r
    g, mg = (dz, mz) if w is None else (dz * w.double(), mz * w.double().abs())
    dx = r * (g - n * (g * n).mean(-1, keepdim=True))
    mag = r * (mg + n.abs() * (mg * n.abs()).mean(-1, keepdim=True))
    dims = (0, 1, 2)
    # dw: chains of the tokens and heads of a thread, then of the blocks
    return ((dx, 2 * NORM * mag + half_step(x.dtype) * dx.abs() + 1e-37),
            ((dz * n).sum(dims), FP32 * (mz * n.abs()).sum(dims) + 1e-37))


class Batch:
    """Sequences with new[b] new tokens and lens[b] keys in all, their pages anywhere in the cache."""

    def __init__(self, new, lens, page, heads, d, dtype, packed=True, seed=0, token_major=False, spare=3, behind=0, width=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        host = torch.Generator().manual_seed(seed)
        self.new, self.len, self.page, self.d, self.dtype = list(new), list(lens), page, d, dtype
        self.H, self.Hkv = heads
        self.packed, B = packed, len(self.new)
        need = [(max(n, 0) + page - 1) // page for n in self.len]
        self.width = max(need + [0]) + 1 if width is None else width
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=host).tolist()
        table = torch.full((B, self.width), -7, dtype=torch.int32)
        for b, n in enumerate(need):
            for e in range(min(n, self.width)):
                table[b, e] = order.pop()
        self.table = table.cuda()
        self.randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dtype)
        shape = (pages, page, self.Hkv, d) if token_major else (pages, self.Hkv, page, d)
        self.K, self.V = (self.randn(*shape).transpose(1, 2) if token_major else self.randn(*shape) for _ in range(2))
        self.lens = torch.tensor(self.len, dtype=torch.int32, device="cuda")
        cu = torch.zeros(B + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(self.new, dtype=torch.int32).cumsum(0)
        self.cu = cu.cuda() if packed else None
        self.rows = (1, int(cu[-1]) + behind) if packed else (B, self.new[0] if B else 0)
        self.Q = self.randn(self.rows[0], self.rows[1], self.H, d).transpose(1, 2)

    @property
    def cache(self):
        return self.K, self.V, self.table

    def place(self, b):
        """Batch row and rows of sequence b."""
        if self.packed:
            r = sum(self.new[:b])
            return 0, slice(r, r + self.new[b])
        return b, slice(0, self.new[b])

    def keys(self, b):
        """Sequence b's K, V [Hkv, len, d] in 64 bits and which of the keys have a page."""
        n = max(self.len[b], 0)
        e = torch.arange(n, device="cuda") // self.page
        slot = torch.arange(n, device="cuda") % self.page
        p = self.table[b].long()[e] if n else e
        there = (p >= 0) & (p < self.K.shape[0])
        p = p.clamp(0, max(self.K.shape[0] - 1, 0))
        return self.K[p, :, slot].transpose(0, 1).double(), self.V[p, :, slot].transpose(0, 1).double(), there

    def visible(self, b, causal=True, window=0):
        n, length = self.new[b], max(self.len[b], 0)
        p = (length - n + torch.arange(n, device="cuda"))[:, None]
        j = torch.arange(length, device="cuda")[None, :]
        see = torch.ones(n, length, dtype=torch.bool, device="cuda") if not causal else j <= p
        return see & (j > p - window) if window else see


def attention(x: Batch, causal=True, window=0, scale=None, sums=False):
    """Per sequence: (O, bound), (lse, bound) [H, n, d] and [H, n] of its new tokens.  sums: the bounds include what the
    scores' own sums may be off by: a chain of d fp32 additions is within d 2^-24 of s sum |q_i k_i|, each
    weight by that power of e, and their sum too (FP32 alone holds for sums of either sign, whose partial ones stay
    small)."""
    u, h = (2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0), half_step(x.dtype)
    s = scale or 1.0 / math.sqrt(x.d)
    g = x.H // x.Hkv
    out = []
    for b in range(len(x.new)):
        row, rows = x.place(b)
        q = x.Q[row, :, rows].double()
        K, V, there = x.keys(b)
        see = x.visible(b, causal, window) & there
        some = see.any(-1)
        # what no token sees has no part, whatever it holds
        used = see.any(0)
        K, V = (torch.where(used[None, :, None], t, torch.zeros_like(t)).repeat_interleave(g, 0) for t in (K, V))
        S = (s * q @ K.transpose(-1, -2)).masked_fill(~see, -math.inf)
        L = torch.logsumexp(S, -1) if S.shape[-1] else torch.full(q.shape[:2], -math.inf, device="cuda", dtype=torch.float64)
        A = torch.where(see, torch.exp(S - torch.where(some, L, torch.zeros_like(L))[..., None]), torch.zeros_like(S))
        O = A @ V
        e = torch.zeros_like(L)[..., None]
        if sums:
            mag = (s * q.abs() @ K.abs().transpose(-1, -2)).masked_fill(~see, 0.0)
            e = x.d * 2.0 ** -24 * mag.amax(-1, keepdim=True)
        tO = (u + FP32 + 2 * e) * (A @ V.abs()) + h * O.abs()
        out.append(((O, tO), (L, FP32 * (1 + L.abs()) + e[..., 0])))
    return out
