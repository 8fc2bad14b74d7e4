"""The paged cache, the attention over it and the normed heads where they can go wrong: layouts of the cache,
offsets past 2^31 elements, streams and captured graphs whose lengths change, many sequences, empty
calls.  References and bounds: tests/paged_reference.py."""
import math

import pytest

from test_gpu_paged import _lib, _t, append_case, attend, batch, dt, randn, tables, within  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------- layouts
def relaid(x, how):
    """The batch's cache in another layout of the same values."""
    torch = _t()
    pages, Hkv, page, d = x.K.shape
    if how == "heads first":      # [Hkv, pages, page, d]
        x.K, x.V = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (x.K, x.V))
    elif how == "interleaved":    # [pages, 2, Hkv, page, d]: one array of both
        both = torch.stack([x.K, x.V], 1).contiguous()
        x.K, x.V = both[:, 0], both[:, 1]
    elif how == "side by side":   # [pages, page, Hkv, 2 d]: a head's key and value in a row
        both = torch.cat([x.K, x.V], -1).transpose(1, 2).contiguous().transpose(1, 2)
        x.K, x.V = both[..., :d], both[..., d:]
    elif how == "unlike":         # K token by token, V head by head
        x.K = x.K.transpose(1, 2).contiguous().transpose(1, 2)
    elif how == "gaps":           # rows, heads and pages apart
        big = torch.zeros(pages, 2 * Hkv, page + 3, d + 16, dtype=x.K.dtype, device="cuda")
        big[:, ::2, :page, :d] = x.K
        x.K = big[:, ::2, :page, :d]
    return x


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["heads first", "interleaved", "side by side", "unlike", "gaps"])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_layouts_of_the_cache(d, how, dtype):
    for new, lens in (([70, 1, 5], [300, 400, 40]), ([1, 1], [333, 64])):
        attend(relaid(batch(new, lens, 32, (4, 2), d, dtype), how))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("page", [16, 48, 80, 112, 192, 256, 1024])
def test_page_sizes(page, dtype):
    for d in (64, 256):
        for new in ([150, 3], [1, 1]):
            attend(batch(new, [700, 260], page, (2, 1), d, dtype), window=0)
            attend(batch(new, [700, 260], page, (2, 1), d, dtype), window=77)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_page_one_head_and_shared_pages(dtype):
    torch = _t()
    x = batch([5], [30], 32, (4, 2), 64, dtype, spare=0)  # a cache of one page
    assert x.K.shape[0] == 1
    attend(x)
    x = batch([40, 1, 1], [200, 200, 130], 16, (3, 1), 128, dtype)
    x.table[1, :8] = x.table[0, :8]                       # a common prefix: the same pages in two rows of the table
    x.table[2, 0:2] = x.table[2, 3]                       # ... and twice in one
    attend(x)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_and_outputs_of_any_strides(dtype):
    torch = _t()
    for d in (64, 128, 256):
        for new in ([40, 3], [1, 1]):
            x = batch(new, [200, 90], 16, (4, 2), d, dtype)
            T = x.rows[1]
            wide = randn(1, T, 7, d + 32, dtype=dt(dtype))
            x.Q = wide[:, :, 1:5, 16:16 + d].transpose(1, 2)          # heads 1 .. 4 of a wider row
            import fwd_bwd_double_gb300 as fbd
            import paged_reference as R
            out = torch.full((1, 4, T + 2, d), 7.0, dtype=dt(dtype), device="cuda")[:, :, :T]   # head by head, with gaps
            O, lse = fbd.attn_paged(x.Q, x.cache, x.lens, x.cu, O=out, max_new=max(new))
            own, _ = fbd.attn_paged(x.Q, x.cache, x.lens, x.cu, max_new=max(new))
            assert own.shape == x.Q.shape and own.stride(2) == 4 * d and torch.equal(own, O)
            for b, (o, L) in enumerate(R.attention(x)):
                r, rows = x.place(b)
                within(O[r, :, rows], o, "O")
                within(lse[r, :, rows], L, "lse")


# ----------------------------------------------------------------------- lengths and scores
@pytest.mark.parametrize("d,heads", [(64, (2, 2)), (128, (4, 1)), (256, (2, 1)), (96, (3, 1))])
def test_long_chunks_shared_by_many_ctas(d, heads):
    for new, lens, window in (([2000], [5000], 0), ([1500, 700], [1500, 6000], 900), ([64], [20000], 0)):
        attend(batch(new, lens, 64, heads, d, "bf16"), window=window)
    attend(batch([700], [2000], 64, heads, d, "bf16"), causal=False)
    attend(batch([300], [1500], 64, heads, d, "f32"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_sequences(dtype):
    import random
    rng = random.Random(5)
    for B, most, heads in ((3000, 1, (2, 1)), (700, 9, (2, 2)), (40, 200, (4, 2))):
        new = [rng.randint(0 if most > 1 else 1, most) for _ in range(B)]
        attend(batch(new, [n + rng.randint(0, 60) for n in new], 16, heads, 64, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_scores_far_apart(d, dtype):
    """Rows whose maximum moves late and by much: keys that grow along the sequence, all products of one sign, so that
    scores reach 3 * 0.64 d / sqrt(d): 31 at d = 256, with log2 e below 2^6, the bound's."""
    torch = _t()
    for new, lens in (([300], [900]), ([1, 1], [900, 400])):
        x = batch(new, lens, 16, (2, 1), d, dtype)
        x.Q = x.Q.abs()
        for b, n in enumerate(lens):
            j = torch.arange(n, device="cuda")
            ramp = (3.0 * j / n)[:, None, None]
            rows = x.K[x.table[b].long()[j // 16], :, j % 16]
            x.K[x.table[b].long()[j // 16], :, j % 16] = (rows.float().abs() * ramp).to(x.K.dtype)
        attend(x, sums=True)
        attend(x, window=200, sums=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_lengths_past_the_table(dtype):
    """lens beyond the table: the keys it lists are held, positions as the lengths say."""
    torch = _t()
    for n in (1, 20):
        x = batch([n, 1], [90, 64], 16, (2, 1), 64, dtype, width=4)       # 64 keys a row of the table
        x.len[0] = 64                                                    # what the reference may see of sequence 0
        import fwd_bwd_double_gb300 as fbd
        import paged_reference as R
        O, lse = fbd.attn_paged(x.Q, x.cache, x.lens, x.cu, causal=False, max_new=n)
        for b, (o, L) in enumerate(R.attention(x, causal=False)):
            r, rows = x.place(b)
            within(O[r, :, rows], o, f"O {b}")
            within(lse[r, :, rows], L, f"lse {b}")


def test_empty_calls_and_caches():
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")     # noqa: E731
    K = z(4, 2, 16, 64)
    for Q, lens, cu in ((z(1, 4, 0, 64), i(3), i(4)), (z(0, 4, 5, 64), i(0), None), (z(1, 4, 5, 64), i(0), i(1))):
        B = lens.shape[0]
        O, lse = fbd.attn_paged(Q, (K, K.clone(), i(B, 2)), lens, cu)
        assert O.shape == Q.shape and lse.shape == Q.shape[:3]
        assert fbd.attn_cache_append(Q[:, :2], Q[:, :2], (K, K.clone(), i(B, 2)), lens, cu) is None
    # a cache without pages, a table without entries: no key anywhere
    for pages, width in ((0, 3), (4, 0), (0, 0)):
        for d in (64, 256):
            for T in (3, 300):
                Kd = z(pages, 2, 16, d)
                cu = torch.tensor([0, T - 1], dtype=torch.int32, device="cuda")
                O, lse = torch.full((1, 4, T, d), 7.0, dtype=torch.bfloat16, device="cuda"), torch.full((1, 4, T), 7.0, device="cuda")
                fbd.attn_paged(z(1, 4, T, d) + 1, (Kd, Kd.clone(), i(1, width)), i(1) + 50, cu, O=O, lse=lse)
                fbd.attn_cache_append(z(1, 2, T, d), z(1, 2, T, d), (Kd, Kd.clone(), i(1, width)), i(1) + 50, cu)
                fbd.attn_device_status()
                assert not O[:, :, :T - 1].any() and (lse[:, :, :T - 1] == -math.inf).all()
                assert (O[:, :, T - 1] == 7.0).all() and (lse[:, :, T - 1] == 7.0).all()


# --------------------------------------------------------------------------- large offsets
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_caches_past_two_to_the_31_elements(dtype):
    """Pages whose elements lie past 2^31 (and, in float32, bytes past 2^33)."""
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    pages, Hkv, page, d = (1 << 31) // (4 * 64 * 128) + 40, 4, 64, 128
    for new, lens in (([1, 1, 1], [300, 64, 129]), ([130, 1, 40], [300, 64, 129])):
        x = batch(new, lens, page, (8, Hkv), d, dtype)
        small = x.K.shape[0]
        K = torch.empty((pages, Hkv, page, d), dtype=dt(dtype), device="cuda")
        assert (pages - small) * Hkv * page * d >= 1 << 31
        V = torch.empty_like(K)
        K[pages - small:], V[pages - small:] = x.K, x.V
        x.K, x.V = K, V
        x.table[x.table >= 0] += pages - small
        attend(x)
        k, v = (x.randn(1, x.rows[1], Hkv, d).transpose(1, 2) for _ in range(2))
        fbd.attn_cache_append(k, v, x.cache, x.lens, x.cu)
        for b in range(len(new)):
            r, rows = x.place(b)
            p = torch.arange(lens[b] - new[b], lens[b], device="cuda")
            where = x.table[b].long()[p // page]
            assert torch.equal(K[where, :, p % page], k[0, :, rows].transpose(0, 1))
            assert torch.equal(V[where, :, p % page], v[0, :, rows].transpose(0, 1))
        del K, V, x


def test_tokens_past_two_to_the_31_elements():
    """Packed tokens, their outputs and the normed heads past 2^31 elements."""
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    H, d, n, page = 128, 128, 125, 16
    B = (1 << 31) // (H * d * n) + 3
    T = B * n
    assert (T - 2 * n) * H * d >= 1 << 31
    Q = torch.zeros((1, T, H, d), dtype=torch.bfloat16, device="cuda")
    x = R.Batch([n], [n + 9], page, (H, 1), d, torch.bfloat16)  # the last sequence; the others see the same pages
    Q[:, T - n:] = x.Q.transpose(1, 2)
    cu = (torch.arange(B + 1, device="cuda") * n).int()
    lens = torch.full((B,), n + 9, dtype=torch.int32, device="cuda")
    O, lse = fbd.attn_paged(Q.transpose(1, 2), (x.K, x.V, x.table.expand(B, -1).contiguous()), lens, cu, max_new=n)
    fbd.attn_device_status()
    (o, L), = R.attention(x)
    within(O[0, :, T - n:], o, "O")
    within(lse[0, :, T - n:], L, "lse")
    del O, lse
    w = 1 + 0.1 * randn(d, dtype=torch.float32)
    y = fbd.attn_qk_norm(Q.transpose(1, 2), w, outs=Q.transpose(1, 2))
    within(y[:, :, T - n:], R.norm(x.Q, w, None), "y")


# ------------------------------------------------------------------------ streams and graphs
def _calls(dtype, d=128):
    """The serving calls of a layer on fixed buffers: append with norm and turn, attention of a chunk and of single
    tokens, the norm and its gradient."""
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    few, many = batch([1] * 9, list(range(100, 1000, 100)), 16, (8, 2), d, dtype), batch([60, 1, 200], [400, 900, 200], 32, (8, 2), d, dtype)
    w = [1 + 0.2 * randn(d, dtype=torch.float32, seed=s) for s in (1, 2)]
    _, freq, axis = tables(1, 1, d, 1)
    k, v = (few.randn(1, few.rows[1], 2, d).transpose(1, 2) for _ in range(2))
    dy = many.randn(1, many.rows[1], 8, d).transpose(1, 2)

    def run():
        q = fbd.attn_cache_append(k, v, few.cache, few.lens, few.cu, Q=few.Q, weights=w, freq=freq, axis=axis)
        a = fbd.attn_paged(q, few.cache, few.lens, few.cu, max_new=1)
        b = fbd.attn_paged(many.Q, many.cache, many.lens, many.cu)
        y = fbd.attn_qk_norm(many.Q, w[0])
        dx, dw = fbd.attn_qk_norm_bwd(many.Q, dy, w[0])
        return [q, *a, *b, y, dx, dw, few.K, few.V]

    return run, few, many


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_two_streams_at_once_and_graphs(dtype):
    """Graphs of the calls on two streams, replayed together over each other, give the eager calls' bits."""
    torch = _t()
    made = [_calls(dtype), _calls(dtype, 64)]
    want = [[t.clone() for t in run()] for run, _, _ in made]
    torch.cuda.synchronize()
    graphs = []
    for run, _, _ in made:
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            run()
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                for _ in range(8):
                    out = run()
        graphs.append((side, g, out))
    for t in (t for _, _, out in graphs for t in out[:-2]):
        t.zero_()
    torch.cuda.synchronize()
    marks = []
    for side, g, _ in graphs:
        with torch.cuda.stream(side):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            for _ in range(10):
                g.replay()
            b.record()
            marks.append((a, b))
    torch.cuda.synchronize()
    assert marks[1][0].elapsed_time(marks[0][1]) > 0 and marks[0][0].elapsed_time(marks[1][1]) > 0  # they overlapped
    for (_, _, out), ref in zip(graphs, want):
        assert all(torch.equal(a, b) for a, b in zip(out, ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_replayed_graph_reads_new_lengths_tables_and_tokens(dtype):
    """The next tokens' graph, replayed as the sequences grow: lengths, table and queries change in place."""
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    for new, hint in (([1, 1, 1], 1), ([40, 3, 150], 0)):
        x = batch(new, [500, 300, 900], 16, (4, 2), 128, dtype)
        cache, lens, cu = tuple(t.clone() for t in x.cache), x.lens.clone(), x.cu.clone()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            fbd.attn_paged(x.Q, cache, lens, cu, max_new=hint)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                O, lse = fbd.attn_paged(x.Q, cache, lens, cu, max_new=hint)
        torch.cuda.synchronize()
        q = x.Q
        for grown, seed in (([17, 901, 350], 1), ([500, 3, 64], 2), ([900, 900, 900], 3)):
            total = [max(a, b) if hint else a for a, b in zip(grown, new)]
            fresh = batch(new, [max(t, 0) for t in total], 16, (4, 2), 128, dtype, seed=seed, width=x.width, spare=200)
            pages = cache[0].shape[0]
            fresh.table[fresh.table >= pages] = -1            # (pages the captured cache does not have)
            fresh.K, fresh.V = fresh.K[:pages], fresh.V[:pages]
            n = fresh.K.shape[0]
            cache[0][:n], cache[1][:n] = fresh.K, fresh.V
            cache[2].copy_(fresh.table), lens.copy_(fresh.lens), q.copy_(fresh.Q)
            fresh.K, fresh.V = cache[0], cache[1]
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for b, (o, L) in enumerate(R.attention(fresh)):
                r, rows = fresh.place(b)
                within(O[r, :, rows], o, f"O {b}")
                within(lse[r, :, rows], L, f"lse {b}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_given_stream_and_workspace(dtype):
    import fwd_bwd_double_gb300 as fbd
    torch = _t()
    x = batch([60, 1, 200], [400, 900, 200], 32, (8, 2), 128, dtype)
    want = [t.clone() for t in fbd.attn_paged(x.Q, x.cache, x.lens, x.cu)]
    desc = fbd.AttnDesc(3, 8, x.rows[1], 128, 0.0, 1, 1 if dtype == "bf16" else 0, 4, 0, None, None)
    ws = torch.full((fbd.attn_paged_workspace_bytes(desc),), 0xff, dtype=torch.uint8, device="cuda")  # NaN
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = fbd.attn_paged(x.Q, x.cache, x.lens, x.cu, workspace=ws, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(fbd.FbdError):
        fbd.attn_paged(x.Q, x.cache, x.lens, x.cu, workspace=ws[:-16])
    w = randn(128, dtype=torch.float32)
    y, (dx, dw) = fbd.attn_qk_norm(x.Q, w), fbd.attn_qk_norm_bwd(x.Q, x.Q, w)
    torch.cuda.synchronize()
    y2, (dx2, dw2) = fbd.attn_qk_norm(x.Q, w, stream=side.cuda_stream), fbd.attn_qk_norm_bwd(x.Q, x.Q, w, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)


# ----------------------------------------------------------------------------- normed heads
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_at_far_positions_and_extreme_sizes(dtype):
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    for d in (32, 256):
        x = randn(1, 2, 40, d, dtype=dt(dtype))
        pos, _, axis = tables(1, 40, d, 2, far=True)
        # whole numbers of steps a turn apart stay exact in 64 bits: frequencies of 2 pi / 2^k
        freq = torch.tensor([2 * math.pi / 2 ** (k % 12) for k in range(d // 2)], device="cuda", dtype=torch.float32)
        p = pos.double()[axis.long().clamp(0, 1)] * freq.double()[:, None, None]
        assert p.abs().max() < 2 ** 34.7                    # their 64-bit products are within 2^-18 of a radian's 2^-1
        y = fbd.attn_qk_norm(x, None, pos, freq, axis)
        r, m = R.norm(x, None, R.cos_sin(pos, freq, axis))
        within(y, (r, m + 2.0 ** -17 * r.abs().amax()), "far")
    for size in (1e15, 1e-15):                              # squares within float32; eps outweighed, then outweighing
        x = (size * randn(1, 2, 40, 64, dtype=torch.float32)).to(dt(dtype))
        w = randn(64, dtype=torch.float32, seed=3)
        within(fbd.attn_qk_norm(x, w), R.norm(x, w, None), f"size {size}")
        dy = randn(1, 2, 40, 64, dtype=dt(dtype), seed=4)
        dx, dw = fbd.attn_qk_norm_bwd(x, dy, w)
        want = R.norm_bwd(x, w, dy, None)
        within(dx, want[0], f"dx {size}")
        within(dw, want[1], f"dw {size}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_norm_gradient_of_many_tokens(dtype):
    """dw over tokens of many blocks; the same bits every time."""
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    for shape in ((3, 7, 2311, 64), (1, 13, 5000, 128), (2, 1, 3001, 32)):
        x, dy = randn(*shape, dtype=dt(dtype)), randn(*shape, dtype=dt(dtype), seed=1)
        w = 1 + 0.2 * randn(shape[-1], dtype=torch.float32, seed=2)
        pos, freq, axis = tables(shape[0], shape[2], shape[3], 2)
        dx, dw = fbd.attn_qk_norm_bwd(x, dy, w, pos, freq, axis)
        want = R.norm_bwd(x, w, dy, R.cos_sin(pos, freq, axis))
        within(dx, want[0], "dx")
        within(dw, want[1], "dw")
        again = fbd.attn_qk_norm_bwd(x, dy, w, pos, freq, axis)
        assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


# --------------------------------------------------------------------------- a few rows
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("n,heads", [(1, (3, 1)), (4, (2, 2)), (2, (6, 2)), (8, (1, 1)), (3, (5, 1)), (4, (8, 2)), (16, (2, 2)), (1, (16, 1))])
def test_few_rows_over_long_contexts(n, heads, d, dtype):
    """Up to 4, 8 and 16 rows (tokens and grouped heads) over contexts of many blocks, of a few keys and of none, with
    pages given up, windows that begin inside a block, and every key visible."""
    new, lens = [n, 1, n, n, 0], [2500, 1, 517, n + 63, 40]
    x = batch(new, lens, 48, heads, d, dtype, behind=3)
    attend(x)
    attend(x, causal=False)
    x.table[0, 3:20] = -1
    x.table[2, 1] = x.K.shape[0]
    attend(x)
    attend(x, window=300)
