"""Latent attention whose second and third loading warps come late (GPU): rows of a few
heads and keys have nothing for them to load, entry after entry, and the ring must not
get ahead of them all the same.  Being late changes no result."""
import numpy as np
import pytest
import torch

from test_gpu_latent import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


def late(pkv, call):
    pkv.set_wait_drill(100_000_000, pkv.DRILL_LATE_PRODUCERS)
    try:
        out = call()
        torch.cuda.synchronize()
    finally:
        pkv.set_wait_drill()
    return out


def short_rows_among_long_ones(n, seed):
    rng = np.random.RandomState(seed)
    return [int(rng.randint(150, 260)) if i % 7 == 6 else int(rng.randint(1, 17)) for i in range(n)]


@pytest.mark.parametrize("H,R,bs", [(8, 512, 16), (8, 256, 16), (1, 512, 32), (8, 512, 64), (130, 256, 16)])
def test_decode_of_short_rows(pkv, H, R, bs):
    c = Case(pkv, "bf16", H, R, 64, short_rows_among_long_ones(700 if H < 100 else 200, H), bs=bs, seed=H)
    want = c.run(pkv)
    assert torch.equal(late(pkv, lambda: c.run(pkv)), want)
    c.check(want, heads=range(0, H, 1 if H < 100 else 43))


@pytest.mark.parametrize("tree", [False, True])
def test_chunks_and_trees(pkv, tree):
    ctx = short_rows_among_long_ones(300, 5)
    C = [int(x) for x in np.random.RandomState(6).randint(0, 5, 300)]
    c = Case(pkv, "bf16", 8, 512, 64, ctx, C, tree, seed=7)
    want = c.run(pkv)
    assert torch.equal(late(pkv, lambda: c.run(pkv)), want)
    c.check(want)


def test_missing_pages(pkv):
    """Tiles of which no page is there: nothing to load for anybody."""
    c = Case(pkv, "bf16", 8, 256, 64, [300, 40] * 100, seed=3)
    c.d_tables[::2, 2:14] = -1
    want = c.run(pkv)
    got = late(pkv, lambda: c.run(pkv))
    assert int(c.status.item()) == pkv.DEV_BAD_BLOCK
    assert torch.equal(got, want)


def test_they_are_late(pkv):
    """A sleep has no least length, so the time is looked at too: 12 entries (two of queries, ten tiles) 10 us each."""
    c = Case(pkv, "bf16", 8, 512, 64, [640] * 300, seed=2)

    def times(n):
        pkv.profile_enable([pkv.KERNEL_LATENT])
        try:
            for _ in range(n):
                c.run(pkv)
            return sorted(1e3 * t for t in pkv.profile_times(pkv.KERNEL_LATENT))
        finally:
            pkv.profile_enable()

    times(3)
    plain = times(11)[5]
    slow = late(pkv, lambda: times(11)[0])
    assert slow > plain + 100, (slow, plain)
