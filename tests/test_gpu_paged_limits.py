"""Calls at the limits of what the paged cache takes: lengths past the table under masks, many small items.  References and
bounds: tests/paged_reference.py."""
import pytest

from test_gpu_paged import _lib, _t, attend, batch, dt  # noqa: F401

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
