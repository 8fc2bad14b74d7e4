"""Differential attention (forward, backward, one token over a cache) and rotary positions
with several axes: the cases they are measured on, their plain forms and their exact values.

A differential head holds two softmax maps over one value head of twice their width:

    A_m = softmax(s Q_m K_m^T + mask),  m = 1, 2;   O = (A_1 - lam_h A_2) V.

Layouts: Q [B, 2H, N, d] and K [B, 2H/g, N, d] with the maps of a head in neighbouring slices
(2h and 2h + 1); V [B, H/g, N, 2d]; O [B, H, N, 2d]; lam [H] float32; g query heads share a
key/value head.  The rotary takes [B, H, N, d] views of any strides and, per pair of
coordinates, a frequency and the position axis it turns with.
"""
import math

import torch

own = False

NEG = float("-inf")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases
def _attn(name, op, B, H, N, d, dtype, mask="causal", g=1, window=0, mean=0):
    return dict(name=name, op=op, B=B, H=H, g=g, N=N, d=d, dtype=dtype, mask=mask, window=window, mean=mean)


def _decode(name, B, H, g, cap, d, dtype, shortest, window=0):
    return dict(name=name, op="decode", B=B, H=H, g=g, cap=cap, d=d, dtype=dtype, shortest=shortest, window=window)


def _rope(name, B, HQ, HK, N, d, dtype, axes, paired, inverse, far):
    return dict(name=name, op="rope", B=B, HQ=HQ, HK=HK, N=N, d=d, dtype=dtype, axes=axes, paired=paired,
                inverse=inverse, far=far)


def listed():
    return [
        # A short prompt's layer in float32, every key visible (an encoder's attention).
        _attn("fwd_short_f32", "fwd", 1, 3, 256, 32, "f32", mask="full"),
        # GPT-2 Small's width (12 maps of 64 columns: six differential heads) at N = 8192, a training batch.
        _attn("fwd_gpt2_n8192", "fwd", 4, 6, 8192, 64, "bf16"),
        # Packed documents of an odd total length, three query heads to a key/value head.
        _attn("fwd_docs_gqa", "fwd", 2, 12, 5001, 64, "bf16", mask="docs", g=3, mean=900),
        # The smallest training step: one short ragged sequence.
        _attn("bwd_short", "bwd", 1, 2, 257, 32, "bf16"),
        # GPT-2 Small's width at N = 4096, a training batch.
        _attn("bwd_gpt2_n4096", "bwd", 4, 6, 4096, 64, "bf16"),
        # A sliding window over one long sequence, shared key/value heads.
        _attn("bwd_window_gqa", "bwd", 1, 12, 8000, 64, "bf16", mask="window", g=4, window=1024),
        # Exact-check precision: float32 gradients.
        _attn("bwd_f32", "bwd", 1, 6, 1000, 64, "f32"),
        # One user's next token on a short context: latency.
        _decode("decode_one_short", 1, 6, 1, 1024, 64, "bf16", 700),
        # A serving batch of ragged contexts, grouped heads.
        _decode("decode_batch_gqa", 32, 16, 4, 8192, 64, "bf16", 100),
        # One very long context, plain heads.
        _decode("decode_one_long", 1, 12, 1, 131072, 64, "bf16", 131000),
        # Positions of video patches (time, height, width) on the queries and keys of a training batch, read
        # from the projection's [B, N, H, d] layout.
        _rope("rope_video_train", 4, 12, 12, 8192, 64, "bf16", 3, "half", False, False),
        # The gradients' turn back, float32, neighbouring pairs, text positions far out.
        _rope("rope_back_f32_far", 2, 8, 4, 1001, 128, "f32", 1, "neighbour", True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "decode", "rope"])
    if op in ("fwd", "bwd"):
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d = rng.choice([32, 64])
        g = rng.choice([1, 1, 2, 3, 4])
        H = g * rng.randint(1, 4)
        N = _log(rng, 1, 6000 if dtype == "bf16" else 1500)
        B = rng.randint(1, 4 if N < 3000 else 2)
        if H * B * N * N > 4 * 6 * 4096 * 4096:
            B = 1
        if H * B * N * N > 4 * 6 * 4096 * 4096:
            N = 4000 + rng.randint(0, 96)
        mask = rng.choice(["causal", "causal", "full", "window", "docs"])
        return dict(op=op, B=B, H=H, g=g, N=N, d=d, dtype=dtype, mask=mask,
                    window=_log(rng, 1, 2000) if mask == "window" else 0,
                    mean=_log(rng, 5, 2000) if mask == "docs" else 0)
    if op == "decode":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        d = rng.choice([32, 64])
        g = rng.choice([1, 2, 4, 8])
        Hkv = rng.randint(1, 8)
        cap = _log(rng, 1, 100000)
        B = max(1, min(64, _log(rng, 1, 64), 1600000 // (Hkv * cap)))
        return dict(op=op, B=B, H=Hkv * g, g=g, cap=cap, d=d, dtype=dtype, shortest=rng.randint(0, cap),
                    window=rng.choice([0, 0, 0, _log(rng, 1, 5000)]))
    N = _log(rng, 1, 20000)
    B = max(1, min(rng.randint(1, 16), 30000 // N))
    HQ = rng.randint(1, 16)
    return dict(op="rope", B=B, HQ=HQ, HK=rng.randint(1, HQ), N=N, d=rng.choice([32, 64, 96, 128]),
                dtype=rng.choice(["bf16", "f32"]), axes=rng.randint(1, 4), paired=rng.choice(["half", "neighbour"]),
                inverse=rng.random() < 0.5, far=rng.random() < 0.3)


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    gen = torch.Generator(device=_device())
    gen.manual_seed(seed)
    return gen


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    gen, dev, dt = _gen(seed), _device(), DT[case["dtype"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    x = {}
    if case["op"] == "rope":
        B, N, d = case["B"], case["N"], case["d"]
        # one projection's output, [B, N, heads, d]: the query heads, then the key heads
        qk = randn(B, N, case["HQ"] + case["HK"], d)
        x["qk"] = qk
        if case["axes"] == 1:
            base = 12000000 if case["far"] else 0
            pos = (base + torch.arange(N, device=dev)).expand(1, B, N)
        else:
            side = max(1, int(round(math.sqrt(N / 8))))
            n = torch.arange(N, device=dev)
            t, h, w = n // (side * side), (n // side) % side, n % side
            rows = [t + (1000000 if case["far"] else 0), h, w, n][:case["axes"]]
            pos = torch.stack(rows).unsqueeze(1).expand(case["axes"], B, N)
        x["pos"] = (pos + torch.randint(0, 50, (1, B, 1), generator=gen, device=dev)).to(torch.int32).contiguous()
        pairs = d // 2
        x["freq"] = (10000.0 ** (-torch.arange(pairs, device=dev, dtype=torch.float64) / pairs)).float()
        # contiguous sections of the pairs, one per axis
        x["axis"] = (torch.arange(pairs, device=dev) * case["axes"] // pairs).to(torch.int32)
        return x
    B, H, g, d = case["B"], case["H"], case["g"], case["d"]
    Hkv = H // g
    x["lam"] = 0.2 + 0.6 * torch.rand(H, generator=gen, device=dev, dtype=torch.float32)
    if case["op"] == "decode":
        cap = case["cap"]
        x["Q"], x["K"], x["V"] = randn(B, 2 * H, 1, d), randn(B, 2 * Hkv, cap, d), randn(B, Hkv, cap, 2 * d)
        x["lens"] = torch.randint(case["shortest"], cap + 1, (B,), generator=gen, device=dev, dtype=torch.int32)
        return x
    N = case["N"]
    x["Q"], x["K"], x["V"] = randn(B, 2 * H, N, d), randn(B, 2 * Hkv, N, d), randn(B, Hkv, N, 2 * d)
    if case["op"] == "bwd":
        x["dO"] = randn(B, H, N, 2 * d)
    if case["mask"] == "docs":
        ends = torch.rand(B, N, generator=gen, device=dev) < 1.0 / max(case["mean"], 1)
        x["seg"] = ends.to(torch.int32).cumsum(1).to(torch.int32).contiguous()
    return x


def _visible(case, x, b, r0, r1):
    """[r1 - r0, N] truth values: which keys the rows r0 .. r1 - 1 of batch row b see."""
    N = case["N"]
    dev = x["Q"].device
    i = torch.arange(r0, r1, device=dev)[:, None]
    j = torch.arange(N, device=dev)[None, :]
    if case["mask"] == "full":
        return torch.ones(r1 - r0, N, dtype=torch.bool, device=dev)
    v = j <= i
    if case["mask"] == "window":
        v = v & (j > i - case["window"])
    if case["mask"] == "docs":
        seg = x["seg"][b]
        v = v & (seg[r0:r1, None] == seg[None, :])
    return v


# ------------------------------------------------------------------------ plain forms
def _softmax(s):
    m = s.max(dim=-1, keepdim=True).values
    e = torch.exp(s - m)
    z = e.sum(dim=-1, keepdim=True)
    return e / z, (m + torch.log(z)).squeeze(-1)


def _maps(x, b, g):
    """Batch row b widened to 32 bits, the key/value heads and the query heads of each as axes of their own:
    q [Hkv, g, 2, N, d], k [Hkv, 1, 2, N, d], v [Hkv, 1, N, 2d]."""
    q, k, v = x["Q"][b].float(), x["K"][b].float(), x["V"][b].float()
    n, N, d = v.shape[0], q.shape[1], q.shape[2]
    return q.view(n, g, 2, N, d), k.view(n, 1, 2, N, d), v.view(n, 1, N, 2 * d)


def _plain_fwd(case, x):
    B, H, g, N, d, dt = case["B"], case["H"], case["g"], case["N"], case["d"], DT[case["dtype"]]
    s = 1.0 / math.sqrt(d)
    dev = x["Q"].device
    O = torch.empty(B, H, N, 2 * d, device=dev, dtype=dt)
    O2 = torch.empty_like(O)
    lse = torch.empty(B, 2 * H, N, device=dev, dtype=torch.float32)
    lam = x["lam"].view(H // g, g, 1, 1)
    for b in range(B):
        hide = ~_visible(case, x, b, 0, N)
        q, k, v = _maps(x, b, g)
        p, L = _softmax((s * (q @ k.transpose(-1, -2))).masked_fill(hide, NEG))
        o = p @ v.unsqueeze(2)                                         # [Hkv, g, 2, N, 2d]
        O[b] = (o[:, :, 0] - lam * o[:, :, 1]).reshape(H, N, 2 * d)
        O2[b] = o[:, :, 1].reshape(H, N, 2 * d)
        lse[b] = L.reshape(2 * H, N)
    return O, O2, lse


def _plain_bwd(case, x):
    B, H, g, N, d, dt = case["B"], case["H"], case["g"], case["N"], case["d"], DT[case["dtype"]]
    s = 1.0 / math.sqrt(d)
    n = H // g
    dQ, dK, dV = torch.empty_like(x["Q"]), torch.empty_like(x["K"]), torch.empty_like(x["V"])
    dlam = torch.zeros_like(x["lam"])
    lam = x["lam"].view(n, g, 1, 1)
    for b in range(B):
        hide = ~_visible(case, x, b, 0, N)
        q, k, v = _maps(x, b, g)
        do = x["dO"][b].float().view(n, g, N, 2 * d)
        dp = do @ v.transpose(-1, -2)                                  # [Hkv, g, N, N]
        p, _ = _softmax((s * (q @ k.transpose(-1, -2))).masked_fill(hide, NEG))
        dV[b] = ((p[:, :, 0] - lam * p[:, :, 1]).transpose(-1, -2) @ do).sum(1)
        delta = (p * dp.unsqueeze(2)).sum(-1, keepdim=True)            # [Hkv, g, 2, N, 1]
        dlam -= delta[:, :, 1].sum((-1, -2)).view(H)
        ds = p * (dp.unsqueeze(2) - delta)
        ds[:, :, 1] *= -lam
        dQ[b] = (s * (ds @ k)).reshape(2 * H, N, d)
        dK[b] = (s * (ds.transpose(-1, -2) @ q)).sum(1).reshape(2 * n, N, d)
    return dQ, dK, dV, dlam


def _plain_decode(case, x):
    B, H, g, cap, d, dt = case["B"], case["H"], case["g"], case["cap"], case["d"], DT[case["dtype"]]
    Hkv = H // g
    s = 1.0 / math.sqrt(d)
    dev = x["Q"].device
    j = torch.arange(cap, device=dev)
    n = x["lens"].long()[:, None]
    see = j < n
    if case["window"]:
        see = see & (j >= n - case["window"])
    see = see[:, None, None, :]                                       # [B, 1, 1, cap]
    q = x["Q"].float().view(B, Hkv, g, 2, d)
    k = x["K"].float().view(B, Hkv, 2, cap, d)
    v = x["V"].float().masked_fill(~see[:, 0, 0, :, None].unsqueeze(1), 0.0)  # [B, Hkv, cap, 2d]
    o = []
    for m in range(2):
        sc = (s * (q[:, :, :, m] @ k[:, :, m].transpose(-1, -2))).masked_fill(~see, NEG)
        top = sc.max(-1, keepdim=True).values
        top = torch.where(top == NEG, torch.zeros_like(top), top)
        e = torch.exp(sc - top)
        z = e.sum(-1, keepdim=True)
        o.append((e @ v) / torch.where(z == 0, torch.ones_like(z), z))
    out = o[0] - x["lam"].view(1, Hkv, g, 1) * o[1]
    return out.reshape(B, H, 1, 2 * d).to(dt)


def _plain_rope(case, x):
    d, dt = case["d"], DT[case["dtype"]]
    p = x["pos"].double()[x["axis"].long()]                           # [pairs, B, N]
    a = p * x["freq"].double()[:, None, None]
    a = a.permute(1, 2, 0)[:, None]                                   # [B, 1, N, pairs]
    c, sn = torch.cos(a).float(), torch.sin(a).float()
    if case["inverse"]:
        sn = -sn
    out = []
    for t in (x["q"], x["k"]):
        t = t.float()
        y = torch.empty(t.shape, device=t.device, dtype=torch.float32)
        if case["paired"] == "half":
            u, v = t[..., :d // 2], t[..., d // 2:]
            y[..., :d // 2], y[..., d // 2:] = u * c - v * sn, u * sn + v * c
        else:
            u, v = t[..., 0::2], t[..., 1::2]
            y[..., 0::2], y[..., 1::2] = u * c - v * sn, u * sn + v * c
        out.append(y.to(dt))
    return tuple(out)


# --------------------------------------------------------------------- prepare and run
def prepare(case, seed):
    x = _inputs(case, seed)
    x["case"] = case
    if case["op"] == "rope":
        # the query and key heads as [B, H, N, d] views of the projection's output
        x["q"] = x["qk"][:, :, :case["HQ"]].transpose(1, 2)
        x["k"] = x["qk"][:, :, case["HQ"]:].transpose(1, 2)
        return x
    if case["op"] == "bwd":  # what the forward pass left
        x["O"], x["O2"], x["lse"] = _plain_fwd(case, x)
    if own and case.get("mask") == "docs":
        import fwd_bwd_double_gb300 as fbd
        x["bounds"] = fbd.attn_segment_bounds(x["seg"])
    return x


def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "decode": _plain_decode, "rope": _plain_rope}[op](case, state)
    import fwd_bwd_double_gb300 as fbd
    x = state
    if op == "rope":
        return tuple(fbd.attn_rope((x["q"], x["k"]), x["pos"], x["freq"], x["axis"], paired=case["paired"],
                                   inverse=case["inverse"]))
    if op == "decode":
        return fbd.attn_diff_decode(x["Q"], x["K"], x["V"], x["lam"], x["lens"], window=case["window"])
    mask = dict(causal=case["mask"] != "full", window=case["window"], bounds=x.get("bounds"))
    if op == "fwd":
        return fbd.attn_diff_fwd(x["Q"], x["K"], x["V"], x["lam"], **mask)
    return fbd.attn_diff_bwd(x["Q"], x["K"], x["V"], x["lam"], x["O"], x["O2"], x["dO"], x["lse"], **mask)


# -------------------------------------------------------------------------------- work
def _pairs(case):
    """Visible (query, key) pairs of one batch row (documents: their mean length)."""
    N = case["N"]
    if case["mask"] == "full":
        return N * N
    reach = N
    if case["mask"] == "window":
        reach = min(N, case["window"])
    if case["mask"] == "docs":
        reach = min(N, case["mean"])
        # documents of geometric length, mean L: a token sees about L keys of its own
        return sum(min(i + 1, reach) for i in range(N))
    return N * (N + 1) // 2 if reach == N else reach * (reach + 1) // 2 + (N - reach) * reach


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"] == "rope":
        n = case["B"] * case["N"] * (case["HQ"] + case["HK"]) * d
        return {"bytes": 2 * n * e + 4 * case["axes"] * case["B"] * case["N"], "flops": 3 * n}
    B, H, g = case["B"], case["H"], case["g"]
    Hkv = H // g
    if case["op"] == "decode":
        keys = B * (case["shortest"] + case["cap"]) // 2
        if case["window"]:
            keys = min(keys, B * case["window"])
        return {"bytes": Hkv * keys * 4 * d * e + B * H * 4 * d * e, "flops": keys * H * 2 * 6 * d}
    N = case["N"]
    q, k = B * H * N * 2 * d * e, B * Hkv * N * 2 * d * e  # both maps' queries (or a value row); keys
    pairs = B * H * _pairs(case)
    if case["op"] == "fwd":  # S_1, S_2 (d each), A_1 V, A_2 V (2d each)
        return {"bytes": q + 2 * k + 2 * q + 8 * B * H * N, "flops": 2 * pairs * 6 * d}
    # S_1, S_2, dQ_m, dK_m (d each), dP and dV once (2d each): dV from the difference of the maps
    return {"bytes": 5 * q + 2 * k + 2 * k + 8 * B * H * N, "flops": 2 * pairs * 10 * d}


# ------------------------------------------------------------------------ exact values
def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits."""
    x = _inputs(case, seed)
    if case["op"] == "rope":
        return _exact_rope(case, x)
    if case["op"] == "decode":
        return _exact_decode(case, x)
    return _exact_attn(case, x)


def _exact_attn(case, x):
    """Rows in blocks; all heads of a key/value group at once; the gradients as the chain
    rule gives them: dA_1 = dO V^T, dA_2 = -lam dO V^T, through each softmax's Jacobian."""
    B, H, g, N, d = case["B"], case["H"], case["g"], case["N"], case["d"]
    Hkv = H // g
    f64 = torch.float64
    Q = x["Q"].to(f64).view(B, Hkv, g, 2, N, d)
    K = x["K"].to(f64).view(B, Hkv, 1, 2, N, d)
    V = x["V"].to(f64).view(B, Hkv, 1, N, 2 * d)
    lam = x["lam"].to(f64).view(Hkv, g)
    bwd = case["op"] == "bwd"
    dO = x["dO"].to(f64).view(B, Hkv, g, N, 2 * d) if bwd else None
    O, O2 = torch.zeros(2, B, Hkv, g, N, 2 * d, dtype=f64, device=Q.device)
    lse = torch.zeros(B, Hkv, g, 2, N, dtype=f64, device=Q.device)
    dQ, dK, dV = torch.zeros_like(Q), torch.zeros_like(K), torch.zeros_like(V)
    dlam = torch.zeros_like(lam)
    step = max(1, min(N, int(2.5e8 / (g * 2 * N))))
    for b in range(B):
        for n in range(Hkv):
            w = torch.stack([torch.ones_like(lam[n]), -lam[n]], 1)[:, :, None, None]  # [g, 2, 1, 1]
            for r in range(0, N, step):
                e = min(N, r + step)
                sc = torch.matmul(Q[b, n, :, :, r:e], K[b, n].transpose(-1, -2)) / math.sqrt(d)
                sc = torch.where(_visible(case, x, b, r, e), sc, torch.full((), NEG, dtype=f64, device=sc.device))
                L = torch.logsumexp(sc, -1)
                A = torch.exp(sc - L[..., None])                      # [g, 2, rows, N]
                if not bwd:
                    om = torch.matmul(A, V[b, n][:, None])
                    O[b, n, :, r:e], O2[b, n, :, r:e], lse[b, n, :, :, r:e] = (w * om).sum(1), om[:, 1], L
                    continue
                dD = torch.matmul(dO[b, n, :, r:e], V[b, n].transpose(-1, -2))[:, None]  # [g, 1, rows, N]
                row = (A * dD).sum(-1, keepdim=True)
                dlam[n] -= row[:, 1].sum((-1, -2))
                J = w * A * (dD - row) / math.sqrt(d)
                dQ[b, n, :, :, r:e] = torch.matmul(J, K[b, n])
                dK[b, n] += torch.matmul(J.transpose(-1, -2), Q[b, n, :, :, r:e]).sum(0, keepdim=True)
                dV[b, n] += torch.matmul((w * A).sum(1).transpose(-1, -2), dO[b, n, :, r:e]).sum(0, keepdim=True)
    if not bwd:
        return O.view(B, H, N, 2 * d), O2.view(B, H, N, 2 * d), lse.view(B, 2 * H, N)
    return dQ.view(B, 2 * H, N, d), dK.view(B, 2 * Hkv, N, d), dV.view(B, Hkv, N, 2 * d), dlam.view(H)


def _exact_decode(case, x):
    B, H, g, d = case["B"], case["H"], case["g"], case["d"]
    out = torch.zeros(B, H, 1, 2 * d, dtype=torch.float64, device=x["Q"].device)
    for b, n in enumerate(x["lens"].tolist()):
        lo = max(0, n - case["window"]) if case["window"] else 0
        if n == lo:
            continue
        K, V = x["K"][b, :, lo:n].double(), x["V"][b, :, lo:n].double()
        for h in range(H):
            a = [torch.softmax(K[2 * (h // g) + m] @ x["Q"][b, 2 * h + m, 0].double() / math.sqrt(d), 0) for m in (0, 1)]
            out[b, h, 0] = (a[0] - x["lam"][h].double() * a[1]) @ V[h // g]
    return out


def _exact_rope(case, x):
    """Each pair as a complex number, turned by its angle."""
    d = case["d"]
    ang = x["freq"].double() * x["pos"].double()[x["axis"].long()].permute(1, 2, 0)   # [B, N, pairs]
    turn = torch.polar(torch.ones_like(ang), -ang if case["inverse"] else ang)[:, :, None]
    t = x["qk"].double()                                                # [B, N, heads, d]
    if case["paired"] == "half":
        z = torch.complex(t[..., :d // 2].contiguous(), t[..., d // 2:].contiguous()) * turn
        y = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_complex(t.reshape(*t.shape[:-1], d // 2, 2).contiguous()) * turn
        y = torch.view_as_real(z).reshape(t.shape)
    y = y.transpose(1, 2)
    return y[:, :case["HQ"]], y[:, case["HQ"]:]
