"""Serving and training operators around attention with normed heads: the RMS norm of each head
with its rotary positions (forward, backward), the append of new keys and values to a paged cache,
and the attention of new tokens over it: the cases they are measured on, their plain forms and
their exact values.

    z = w x / sqrt(mean x^2 + eps),  y = z turned by its position            (attn_qk_norm)
    the same for the new keys (and queries), written to the cache's pages     (attn_cache_append)
    O = softmax(s Q K^T + mask) V over a sequence's pages, lse                (attn_paged)

Layouts: queries and keys are [B, H, N, d] views of a projection's [B, N, heads, d] output; packed
tokens [1, H, T, d] with the sequences' first rows cu [B + 1]; a cache's K and V are
[pages, Hkv, page, d] with a table [B, width] of each sequence's pages and lens [B], the keys it
holds, the new tokens' among them.
"""
import math

import torch

own = False

NEG = float("-inf")
EPS = 1e-6
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases
def _norm(name, op, B, N, HQ, HK, d, dtype, axes=1, paired="half"):
    return dict(name=name, op=op, B=B, N=N, HQ=HQ, HK=HK, d=d, dtype=dtype, axes=axes, paired=paired)


def _cache(name, op, B, H, g, d, dtype, page, new_lo, new_hi, ctx_lo, ctx_hi, mask="causal", window=0, norm=True,
           token_major=False):
    """B sequences with new_lo .. new_hi new tokens each behind ctx_lo .. ctx_hi keys in the cache."""
    return dict(name=name, op=op, B=B, H=H, g=g, d=d, dtype=dtype, page=page, new_lo=new_lo, new_hi=new_hi,
                ctx_lo=ctx_lo, ctx_hi=ctx_hi, mask=mask, window=window, norm=norm, token_major=token_major)


def listed():
    return [
        # The queries and keys of a training batch at GPT-2 Small's width, from the projection's layout.
        _norm("norm_gpt2_n8192", "norm", 4, 8192, 12, 12, 64, "bf16"),
        # Their gradients, the weights' among them.
        _norm("norm_bwd_gpt2_n8192", "norm_bwd", 4, 8192, 12, 12, 64, "bf16"),
        # Exact-check precision on a short video clip: three axes, an odd length, neighbouring pairs.
        _norm("norm_bwd_short_f32", "norm_bwd", 2, 257, 6, 2, 96, "f32", 3, "neighbour"),
        # A prompt batch's keys, values and queries, grouped heads, pages of 64.
        _cache("append_prompts", "append", 8, 16, 4, 128, "bf16", 64, 500, 4000, 0, 300),
        # One new token of each sequence of a serving batch: latency.
        _cache("append_one_each", "append", 32, 12, 1, 64, "bf16", 16, 1, 1, 10, 2000),
        # A short follow-up on a short context: the smallest chunk.
        _cache("chunk_short", "paged", 1, 6, 1, 64, "bf16", 16, 16, 16, 200, 200),
        # The last 8192 tokens of a long prompt over the pages written before.
        _cache("chunk_long", "paged", 1, 16, 4, 128, "bf16", 64, 8192, 8192, 24000, 24000),
        # Prompts and follow-ups of ragged lengths in one batch, a sliding window, pages of 48 laid out
        # token by token.
        _cache("chunk_ragged_window", "paged", 12, 12, 3, 96, "bf16", 48, 1, 1500, 0, 9000, window=2000, token_major=True),
        # Wide heads, every key visible (a prompt read in both directions).
        _cache("chunk_wide_full", "paged", 2, 8, 2, 256, "bf16", 128, 1000, 1000, 3000, 4000, mask="full"),
        # Exact-check precision.
        _cache("chunk_f32", "paged", 3, 6, 2, 64, "f32", 32, 100, 400, 0, 1500),
        # The next token of each sequence of a serving batch, ragged contexts, grouped heads.
        _cache("token_batch", "paged", 64, 32, 8, 128, "bf16", 16, 1, 1, 100, 8191),
        # The next token of one very long context.
        _cache("token_long", "paged", 1, 16, 4, 128, "bf16", 64, 1, 1, 131000, 131000),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "append", "paged", "paged", "paged"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    d = rng.choice([32, 64, 96, 128, 256])
    if op in ("norm", "norm_bwd"):
        N = _log(rng, 1, 20000)
        B = max(1, min(rng.randint(1, 16), 20000 // N))
        HQ = rng.randint(1, 12)
        HK = rng.randint(1, HQ)
        N = max(1, min(N, 32768 * 24 * 64 // (B * (HQ + HK) * d)))
        return dict(op=op, B=B, N=N, HQ=HQ, HK=HK, d=d, dtype=dtype, axes=rng.randint(1, 4),
                    paired=rng.choice(["half", "neighbour"]))
    g = rng.choice([1, 2, 3, 4, 5, 8])
    Hkv = rng.randint(1, 6)
    case = dict(op=op, H=g * Hkv, g=g, d=d, dtype=dtype, page=rng.choice([16, 32, 48, 64, 128, 256]),
                token_major=rng.random() < 0.3, mask="causal", window=0, norm=rng.random() < 0.7)
    if op == "append":
        new_hi = _log(rng, 1, 4000)
        case.update(B=max(1, min(_log(rng, 1, 64), 24000 // new_hi)), new_lo=rng.randint(0, new_hi), new_hi=new_hi, ctx_lo=0,
                    ctx_hi=_log(rng, 1, 3000))
        return case
    kind = rng.choice(["token", "few", "chunk"])
    if kind == "token":
        new_lo, new_hi = 1, 1
        ctx_hi = _log(rng, 1, 100000)
        B = max(1, min(_log(rng, 1, 96), 1500000 // (Hkv * ctx_hi)))
    elif kind == "few":
        new_hi = rng.randint(1, 40)
        new_lo = rng.randint(0, new_hi)
        ctx_hi = _log(rng, 1, 30000)
        B = max(1, min(_log(rng, 1, 32), 400000 // (Hkv * ctx_hi)))
    else:
        new_hi = _log(rng, 16, 4000 if dtype == "bf16" else 1000)
        new_lo = rng.randint(0, new_hi)
        ctx_hi = _log(rng, 1, 20000 if dtype == "bf16" else 4000)
        B = max(1, min(rng.randint(1, 8), 30000 * 4000 // (new_hi * (ctx_hi + new_hi))))
    if dtype == "f32" and kind != "chunk":
        ctx_hi = max(1, ctx_hi // 4)
    case.update(B=B, new_lo=new_lo, new_hi=new_hi, ctx_lo=rng.randint(0, ctx_hi), ctx_hi=ctx_hi,
                mask=rng.choice(["causal", "causal", "full"]))
    if case["mask"] == "causal" and rng.random() < 0.3:
        case["window"] = _log(rng, 1, 5000)
    return case


# ----------------------------------------------------------------------------- inputs
def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _new(case):
    """The new tokens of each sequence: a case's own, so that its shapes are too."""
    gen = torch.Generator().manual_seed(case["B"] * 100003 + case["new_hi"])
    return torch.randint(case["new_lo"], case["new_hi"] + 1, (case["B"],), generator=gen)


def _inputs(case, seed):
    """The tensors of a case, from the seed alone."""
    dev, dt, d = _device(), DT[case["dtype"]], case["d"]
    gen = torch.Generator(device=dev).manual_seed(seed)
    host = torch.Generator().manual_seed(seed)  # the sequences' lengths, which a server knows on the host

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).to(dt)

    def weight():
        return 1.0 + 0.2 * torch.randn(d, generator=gen, device=dev, dtype=torch.float32)

    x = {"wq": weight(), "wk": weight()}
    pairs = d // 2
    x["freq"] = (10000.0 ** (-torch.arange(pairs, device=dev, dtype=torch.float64) / pairs)).float()
    if case["op"] in ("norm", "norm_bwd"):
        B, N, axes = case["B"], case["N"], case["axes"]
        x["axis"] = (torch.arange(pairs, device=dev) * axes // pairs).to(torch.int32)  # sections of the pairs
        side = max(1, int(round(math.sqrt(N / 8))))
        n = torch.arange(N, device=dev)
        rows = [n] if axes == 1 else [n // (side * side), (n // side) % side, n % side, n][:axes]
        start = torch.randint(0, 50, (1, B, 1), generator=gen, device=dev)
        x["pos"] = (torch.stack(rows).unsqueeze(1) + start).to(torch.int32).contiguous()
        x["qk"] = 1.5 * randn(B, N, case["HQ"] + case["HK"], d)
        if case["op"] == "norm_bwd":
            x["dy"] = [randn(B, h, N, d) for h in (case["HQ"], case["HK"])]
        return x
    B, H, g, page = case["B"], case["H"], case["g"], case["page"]
    Hkv = H // g
    new = _new(case)
    lens = new + torch.randint(case["ctx_lo"], case["ctx_hi"] + 1, (B,), generator=host)
    need = (lens + page - 1) // page
    width = (case["ctx_hi"] + case["new_hi"] + page - 1) // page
    pages = B * width
    order = torch.randperm(pages, generator=host).tolist()  # a sequence's pages lie anywhere
    table = torch.full((B, width), -1, dtype=torch.int32)
    for b, n in enumerate(need.tolist()):
        table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    cu = torch.zeros(B + 1, dtype=torch.int32)
    cu[1:] = new.cumsum(0)
    T = max(int(cu[-1]), 1)
    x.update(new=new.tolist(), len=lens.tolist(), cu=cu.to(dev), lens=lens.to(torch.int32).to(dev), table=table.to(dev))
    x["axis"] = torch.zeros(pairs, dtype=torch.int32, device=dev)
    for name in ("K", "V"):
        if case["token_major"]:
            x[name] = randn(pages, page, Hkv, d).transpose(1, 2)
        else:
            x[name] = randn(pages, Hkv, page, d)
    # one projection's output, [T, heads, d]: queries, then (for the append) the new keys and values
    x["qkv"] = 1.5 * randn(1, T, H + (2 * Hkv if case["op"] == "append" else 0), d)
    if case["op"] == "paged":
        x["qkv"] = x["qkv"] / 1.5
    return x


# ------------------------------------------------------------------------ plain forms
def _angles(pos, freq, axis):
    """cos, sin [..., tokens, pairs] in 32 bits of freq[i] pos[axis[i]] formed in 64; pos [axes, ..., tokens]."""
    a = (pos.double()[axis.long()] * freq.double().view(-1, *([1] * (pos.dim() - 1)))).movedim(0, -1)
    return torch.cos(a).float(), torch.sin(a).float()


def _pairs(t, paired):
    d = t.shape[-1]
    return (t[..., :d // 2], t[..., d // 2:]) if paired == "half" else (t[..., 0::2], t[..., 1::2])


def _turn(t, c, s, paired):
    u, v = _pairs(t, paired)
    y = torch.empty_like(t)
    a, b = _pairs(y, paired)
    a.copy_(u * c - v * s)
    b.copy_(u * s + v * c)
    return y


def _rms(t, w):
    """t in 32 bits, [..., d]: its norm and 1 / rms."""
    r = torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)
    return t * r * w, r


def _plain_norm(case, x):
    dt = DT[case["dtype"]]
    c, s = (t[:, None] for t in _angles(x["pos"], x["freq"], x["axis"]))         # [B, 1, N, pairs]
    return tuple(_turn(_rms(t.float(), w)[0], c, s, case["paired"]).to(dt)
                 for t, w in ((x["q"], x["wq"]), (x["k"], x["wk"])))


def _plain_norm_bwd(case, x):
    dt = DT[case["dtype"]]
    c, s = (t[:, None] for t in _angles(x["pos"], x["freq"], x["axis"]))
    dxs, dws = [], []
    for t, w, dy in ((x["q"], x["wq"], x["dy"][0]), (x["k"], x["wk"], x["dy"][1])):
        t = t.float()
        dz = _turn(dy.float(), c, -s, case["paired"])
        _, r = _rms(t, w)
        n = t * r
        dws.append((dz * n).sum((0, 1, 2), dtype=torch.float64).float())
        h = dz * w
        dxs.append((r * (h - n * (h * n).mean(-1, keepdim=True))).to(dt))
    return dxs[0], dxs[1], dws[0], dws[1]


def _slots(case, x):
    """Per packed token: its position in its sequence, its page and its slot there."""
    cu, lens = x["cu"].long(), x["lens"].long()
    n = cu[1:] - cu[:-1]
    seq = torch.repeat_interleave(torch.arange(case["B"], device=cu.device), n)
    pos = torch.arange(seq.numel(), device=cu.device) - cu[seq] + (lens - n)[seq]
    return pos, x["table"].long()[seq, pos // case["page"]], pos % case["page"]


def _plain_append(case, x):
    dt = DT[case["dtype"]]
    pos, page, slot = _slots(case, x)
    T = pos.numel()
    c, s = _angles(pos[None], x["freq"], x["axis"])                               # [T, pairs]
    q, k, v = (x[name][0, :, :T].float() for name in ("q", "k", "v"))             # [heads, T, d]
    if case["norm"]:
        q, k = _rms(q, x["wq"])[0], _rms(k, x["wk"])[0]
    x["K"][page, :, slot] = _turn(k, c, s, "half").to(dt).transpose(0, 1)
    x["V"][page, :, slot] = v.to(dt).transpose(0, 1)
    out = torch.zeros(x["q"].shape, dtype=dt, device=q.device)
    out[0, :, :T] = _turn(q, c, s, "half").to(dt)
    return out, x["K"], x["V"]


def _visible(case, start, t0, t1, length, dev):
    p = start + torch.arange(t0, t1, device=dev)[:, None]
    j = torch.arange(length, device=dev)[None, :]
    if case["mask"] == "full":
        return torch.ones(t1 - t0, length, dtype=torch.bool, device=dev)
    see = j <= p
    return see & (j > p - case["window"]) if case["window"] else see


def _plain_paged(case, x):
    dt, d, g = DT[case["dtype"]], case["d"], case["g"]
    q = x["q"]
    H, T = q.shape[1], q.shape[2]
    dev = q.device
    O = torch.zeros(1, H, T, d, dtype=dt, device=dev)
    lse = torch.zeros(1, H, T, dtype=torch.float32, device=dev)
    row = 0
    for b, (n, length) in enumerate(zip(x["new"], x["len"])):
        if n == 0:
            continue
        used = x["table"][b, :(length + case["page"] - 1) // case["page"]].long()
        hide = ~_visible(case, length - n, 0, n, length, dev)
        for h in range(H // g):
            k = x["K"][used, h].reshape(-1, d)[:length].float()
            v = x["V"][used, h].reshape(-1, d)[:length].float()
            sc = (q[0, h * g:(h + 1) * g, row:row + n].float() @ k.transpose(0, 1)) * (1.0 / math.sqrt(d))
            sc = sc.masked_fill(hide, NEG)
            m = sc.max(-1, keepdim=True).values
            e = torch.exp(sc - m)
            z = e.sum(-1, keepdim=True)
            O[0, h * g:(h + 1) * g, row:row + n] = ((e @ v) / z).to(dt)
            lse[0, h * g:(h + 1) * g, row:row + n] = (m + torch.log(z))[..., 0]
        row += n
    return O, lse


# --------------------------------------------------------------------- prepare and run
def prepare(case, seed):
    x = _inputs(case, seed)
    x["case"] = case
    if case["op"] in ("norm", "norm_bwd"):
        x["q"], x["k"] = (t.transpose(1, 2) for t in x["qk"].split([case["HQ"], case["HK"]], 2))
        return x
    H, Hkv = case["H"], case["H"] // case["g"]
    if case["op"] == "append":
        x["q"], x["k"], x["v"] = (t.transpose(1, 2) for t in x["qkv"].split([H, Hkv, Hkv], 2))
        x["out"] = torch.zeros(x["q"].shape, dtype=x["q"].dtype, device=x["q"].device)
    else:
        x["q"] = x["qkv"].transpose(1, 2)
        # a program keeps its output buffers; rows of no sequence stay as they were
        x["O"] = torch.zeros_like(x["q"])
        x["lse"] = torch.zeros(x["q"].shape[:3], dtype=torch.float32, device=x["q"].device)
    return x


def run(state):
    x = state
    case = x["case"]
    op = case["op"]
    if not own:
        return {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "append": _plain_append, "paged": _plain_paged}[op](case, x)
    import fwd_bwd_double_gb300 as fbd
    if op == "norm":
        return tuple(fbd.attn_qk_norm((x["q"], x["k"]), (x["wq"], x["wk"]), x["pos"], x["freq"], x["axis"],
                                      paired=case["paired"], eps=EPS))
    if op == "norm_bwd":
        dxs, dws = fbd.attn_qk_norm_bwd((x["q"], x["k"]), x["dy"], (x["wq"], x["wk"]), x["pos"], x["freq"], x["axis"],
                                        paired=case["paired"], eps=EPS)
        return (*dxs, *dws)
    cache = (x["K"], x["V"], x["table"])
    if op == "append":
        weights = (x["wq"], x["wk"]) if case["norm"] else None
        fbd.attn_cache_append(x["k"], x["v"], cache, x["lens"], x["cu"], Q=x["q"], Q_out=x["out"], weights=weights,
                              freq=x["freq"], axis=x["axis"], eps=EPS)
        return x["out"], x["K"], x["V"]
    return fbd.attn_paged(x["q"], cache, x["lens"], x["cu"], O=x["O"], lse=x["lse"], causal=case["mask"] == "causal",
                          window=case["window"], max_new=case["new_hi"])


# -------------------------------------------------------------------------------- work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    d = case["d"]
    if case["op"] in ("norm", "norm_bwd"):
        tokens = case["B"] * case["N"]
        n = tokens * (case["HQ"] + case["HK"]) * d
        if case["op"] == "norm":
            return {"bytes": 2 * n * e + 4 * case["axes"] * tokens, "flops": 7 * n}
        return {"bytes": 3 * n * e + 4 * case["axes"] * tokens, "flops": 15 * n}
    B, H, g = case["B"], case["H"], case["g"]
    Hkv = H // g
    news = _new(case).tolist()
    ctx = (case["ctx_lo"] + case["ctx_hi"]) / 2
    if case["op"] == "append":
        n = sum(news) * (H + 2 * Hkv) * d
        return {"bytes": 2 * n * e, "flops": 7 * n}
    keys = pairs = 0  # that some token of a sequence sees; visible (token, key) pairs: at the mean context
    for new in news:
        if case["mask"] == "full":
            mean, seen = ctx + new, ctx + new
        else:
            mean, seen = ctx + (new + 1) / 2, ctx + new
            if case["window"]:
                mean, seen = min(mean, case["window"]), min(seen, case["window"] + new)
        keys += seen if new else 0
        pairs += new * mean
    rows = sum(news) * H
    return {"bytes": int(2 * Hkv * keys * d * e + 2 * rows * d * e + 4 * rows), "flops": int(4 * H * pairs * d)}


# ------------------------------------------------------------------------ exact values
def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits."""
    x = _inputs(case, seed)
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "append": _exact_append, "paged": _exact_paged}[case["op"]](case, x)


def _complex(t, paired):
    """[..., d] as d / 2 complex numbers, one per pair."""
    d = t.shape[-1]
    if paired == "half":
        return torch.complex(t[..., :d // 2].contiguous(), t[..., d // 2:].contiguous())
    return torch.view_as_complex(t.reshape(*t.shape[:-1], d // 2, 2).contiguous())


def _real(z, paired):
    return torch.cat([z.real, z.imag], -1) if paired == "half" else torch.view_as_real(z).flatten(-2)


def _turns(pos, freq, axis):
    """exp(i freq pos) [..., tokens, pairs] of pos [axes, ..., tokens]."""
    ang = torch.movedim(pos.double()[axis.long()], 0, -1) * freq.double()
    return torch.polar(torch.ones_like(ang), ang)


def _exact_norm(case, x):
    z = x["qk"].double()                                                          # [B, N, heads, d]
    z = z / torch.sqrt(z.square().mean(-1, keepdim=True) + EPS)
    HQ = case["HQ"]
    z = torch.cat([z[:, :, :HQ] * x["wq"].double(), z[:, :, HQ:] * x["wk"].double()], 2)
    turn = _turns(x["pos"], x["freq"], x["axis"])[:, :, None]
    y = _real(_complex(z, case["paired"]) * turn, case["paired"]).transpose(1, 2)
    return y[:, :HQ], y[:, HQ:]


def _exact_norm_bwd(case, x):
    """By the chain rule on norms: with u = x / rms, dx = (g - u <g, u> / d) / rms, g = w dz."""
    turn = _turns(x["pos"], x["freq"], x["axis"])[:, None].conj()                 # [B, 1, N, pairs]
    dxs, dws = [], []
    for t, dy, w in zip(x["qk"].split([case["HQ"], case["HK"]], 2), x["dy"], (x["wq"], x["wk"])):
        t = t.transpose(1, 2).double()
        rms = (t.square().sum(-1, keepdim=True) / case["d"] + EPS).sqrt()
        dz = _real(_complex(dy.double(), case["paired"]) * turn, case["paired"])
        u = t / rms
        dws.append(torch.einsum("bhnd,bhnd->d", dz, u))
        gr = dz * w.double()
        dxs.append((gr - u * (torch.einsum("bhnd,bhnd->bhn", gr, u)[..., None] / case["d"])) / rms)
    return dxs[0], dxs[1], dws[0], dws[1]


def _exact_append(case, x):
    B, H, page = case["B"], case["H"], case["page"]
    Hkv = H // case["g"]
    K, V = x["K"].double(), x["V"].double()
    qkv = x["qkv"][0].double()                                                    # [T, heads, d]
    out = torch.zeros(1, H, qkv.shape[0], case["d"], dtype=torch.float64, device=qkv.device)
    row = 0
    for b, (n, length) in enumerate(zip(x["new"], x["len"])):
        if n == 0:
            continue
        p = torch.arange(length - n, length, device=qkv.device)
        t = qkv[row:row + n]
        qk = t[:, :H + Hkv]
        if case["norm"]:
            qk = qk / torch.sqrt(qk.square().mean(-1, keepdim=True) + EPS)
            qk = torch.cat([qk[:, :H] * x["wq"].double(), qk[:, H:] * x["wk"].double()], 1)
        qk = _real(_complex(qk, "half") * _turns(p[None], x["freq"], x["axis"])[:, None], "half")
        out[0, :, row:row + n] = qk[:, :H].transpose(0, 1)
        where = x["table"][b].long()[torch.div(p, page, rounding_mode="floor")]
        K[where, :, p % page] = qk[:, H:]
        V[where, :, p % page] = t[:, H + Hkv:]
        row += n
    return out, K, V


def _exact_paged(case, x):
    """Sequence by sequence, a few rows at a time, all query heads of a key/value head at once."""
    g, d, page = case["g"], case["d"], case["page"]
    q = x["qkv"][0].double()                                                      # [T, H, d]
    T, H = q.shape[:2]
    O = torch.zeros(1, H, T, d, dtype=torch.float64, device=q.device)
    lse = torch.zeros(1, H, T, dtype=torch.float64, device=q.device)
    row = 0
    for b, (n, length) in enumerate(zip(x["new"], x["len"])):
        if n == 0:
            continue
        pos = torch.arange(length, device=q.device)
        where, slot = x["table"][b].long()[torch.div(pos, page, rounding_mode="floor")], pos % page
        step = max(1, min(n, int(2e8 / (g * length))))
        for h in range(H // g):
            K, V = x["K"][where, h, slot].double(), x["V"][where, h, slot].double()
            for t in range(0, n, step):
                e = min(n, t + step)
                Q = q[row + t:row + e, h * g:(h + 1) * g].transpose(0, 1) / math.sqrt(d)   # [g, rows, d]
                sc = torch.where(_visible(case, length - n, t, e, length, q.device), torch.matmul(Q, K.T),
                                 torch.full((), NEG, dtype=torch.float64, device=q.device))
                L = torch.logsumexp(sc, -1)
                O[0, h * g:(h + 1) * g, row + t:row + e] = torch.matmul(torch.exp(sc - L[..., None]), V)
                lse[0, h * g:(h + 1) * g, row + t:row + e] = L
        row += n
    return O, lse
