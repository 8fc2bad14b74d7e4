"""Calls at the limits of what the paged cache takes: lengths past the table under masks, many small items,
sequences by the million.  References and bounds: tests/paged_reference.py."""
import pytest

from test_gpu_paged import _lib, _t, attend, batch, dt, within  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- lengths past the table, windows
def past_the_table(new, lens, page, width, heads, d, dtype, **kw):
    """Sequences whose lengths may pass width * page keys: positions as the lengths say, the table's keys held."""
    import paged_reference as R
    torch = _t()

    class Past(R.Batch):
        def held(self, b):
            return min(max(self.len[b], 0), self.width * self.page)

        def keys(self, b):
            n = self.len[b]
            self.len[b] = self.held(b)
            try:
                return super().keys(b)
            finally:
                self.len[b] = n

        def visible(self, b, causal=True, window=0):
            n = self.new[b]
            p = (max(self.len[b], 0) - n + torch.arange(n, device="cuda"))[:, None]
            j = torch.arange(self.held(b), device="cuda")[None, :]
            see = j <= p if causal else torch.ones(n, self.held(b), dtype=torch.bool, device="cuda")
            return see & (j > p - window) if window else see

    return Past(new, lens, page, heads, d, dt(dtype), width=width, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 20, 150])
def test_windows_of_lengths_past_the_table(n, d, dtype):
    """A window as wide as the table (64 keys) or wider still hides keys from a token behind the table's end: of lens 90,
    the token at 89 sees 26 .. 63 under a window of 64, and none of the last sequence's 64 keys is in sight of it."""
    x = past_the_table([n, n, n, n], [90, 64, 63 + n, 129 + n], 16, 4, (4, 2), d, dtype)
    for window in (0, 1, 30, 63, 64, 65, 89, 90, 128, 1000, (1 << 31) - 1, 1 << 40):
        attend(x, window=window)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_windows_near_the_largest_length(dtype):
    """Positions next to 2^31: their differences with a window leave 32 bits nowhere."""
    top = (1 << 31) - 1
    for n in (1, 40):
        x = past_the_table([n, n], [90, 90], 16, 8, (4, 2), 64, dtype)
        x.len[0] = top
        x.lens[0] = top
        for window in (0, 100, top - 60, top - 1, top):
            attend(x, window=window)


# --------------------------------------------------------------------- items of few key blocks
@pytest.mark.parametrize("d,heads", [(64, (4, 4)), (128, (8, 2)), (96, (3, 1))])
def test_many_items_of_two_and_three_blocks(d, heads):
    """Items of one tile over one, two and three blocks of 128 keys, tens of them a CTA one after another: the second half
    of each is joined to the first while the next ones are under way."""
    import random
    rng = random.Random(7)
    new = [rng.randint(17, 40) for _ in range(900)]
    lens = [n + rng.choice([0, 60, 130, 200, 230, 300, 340]) for n in new]
    x = batch(new, lens, 32, heads, d, "bf16")
    attend(x)
    attend(x, window=90)


# ------------------------------------------------------------------------ very many sequences
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("n", [1, 30])
def test_a_few_tokens_among_the_most_sequences(n, d, dtype):
    """New tokens of a few sequences among 2^25 - 1, the most that a call takes: the first and the last one follow one another
    in a CTA's stretch, and what lies between is passed within the waits' bounds."""
    import fwd_bwd_double_gb300 as fbd
    import paged_reference as R
    torch = _t()
    B = (1 << 25) - 1
    for where in ([0, B - 1], [0, 1, B // 2, B - 2, B - 1]):
        x = batch([n] * len(where), [n + 20 * k for k in range(len(where))], 64, (1, 1), d, dtype, width=2)
        at = torch.tensor(where, device="cuda")
        new = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
        new[at + 1] = n
        cu = new.cumsum(0, dtype=torch.int32)
        lens = torch.full((B,), 9, dtype=torch.int32, device="cuda")
        table = torch.full((B, 2), -1, dtype=torch.int32, device="cuda")
        lens[at], table[at] = x.lens, x.table
        O, lse = torch.full_like(x.Q, 7.0), torch.full(x.Q.shape[:3], 7.0, device="cuda")
        fbd.attn_paged(x.Q, (x.K, x.V, table), lens, cu, O=O, lse=lse, max_new=n)
        fbd.attn_device_status()
        for b, (o, L) in enumerate(R.attention(x)):
            r, rows = x.place(b)
            within(O[r, :, rows], o, f"O of sequence {where[b]}")
            within(lse[r, :, rows], L, f"lse of sequence {where[b]}")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_runs_of_empty_sequences(dtype):
    """Empty sequences in runs of every length around the 32 and 128 that are passed at once, in front and behind too."""
    for runs in ([0, 1, 30, 31, 32, 33, 95, 96, 97], [127, 128, 129, 255, 256, 257, 500], [31, 127, 0, 0, 160]):
        new = []
        for k, r in enumerate(runs):
            new += [0] * r + [1 + k % 3]
        new += [0] * runs[-1]
        lens = [v + (7 * i) % 40 if v else i % 50 for i, v in enumerate(new)]
        x = batch(new, lens, 16, (1, 1), 64, dtype)
        attend(x)
        attend(x, max_new=0)
        attend(batch(new, lens, 16, (1, 1), 256, dtype), max_new=0)
