"""Forks and rollbacks where a block has expired or none is free: the library and
the reference model alike."""
import pytest

from oracle.allocator_model import AllocatorModel, OutOfBlocks
from test_allocator_pages import Lib


@pytest.fixture(params=["model", "library"])
def make(request):
    if request.param == "model":
        class M(AllocatorModel):
            def refs(self, n):
                return self.refcount[:n]
        return M
    import block_paged_kv_gb300 as pkv
    return lambda *a: Lib(pkv, *a)


@pytest.mark.parametrize("call", ["fork", "truncate"])
@pytest.mark.parametrize("n", [5, 7, 22, 23])
def test_an_expired_place_is_refused(make, call, n):
    m = make(4, 16, 16)
    r = m.begin()
    m.reserve(r, 40)
    m.expire_window(r, 24, 4)                       # blocks 1 .. 5 are gone, the sinks' stays
    before = (m.table(r), m.refs(16), m.stats())
    with pytest.raises(OutOfBlocks):                # token n could never be stored
        getattr(m, call)(r, n)
    assert (m.table(r), m.refs(16), m.stats()) == before


@pytest.mark.parametrize("n", [3, 4, 24, 26])
def test_places_beside_the_expired_ones_are_not(make, n):
    m = make(4, 16, 16)
    r = m.begin()
    m.reserve(r, 40)
    m.expire_window(r, 24, 4)
    c, copy = m.fork(r, n)
    want = [0] + [-1] * 5
    assert m.table(c)[:n // 4] == want[:n // 4]
    assert copy == (None if n % 4 == 0 else ({3: 0, 26: 6}[n], 1))   # block 1 is the lowest free one
    assert m.truncate(r, n) is None
    for q in (r, c):
        m.reserve(q, n + 1)                         # token n has a block
        assert m.table(q)[n // 4] >= 0


def test_a_rollback_evicts_and_grows_nothing_while_it_frees_blocks(make):
    m = make(4, 5, 10)
    s = m.begin()
    m.reserve(s, 4)
    m.publish(s, [9] * 4)
    m.release(s)                                    # block 0 cached
    r, toks = m.begin(), list(range(16))
    m.reserve(r, 16)                                # blocks 1 .. 4: none is free now
    m.publish(r, toks[:8])                          # 1, 2 published, 3 and 4 private
    assert m.truncate(r, 7) == (2, 3)               # 3 goes with the rollback: it holds the copy
    assert m.table(r) == [1, 3] and m.refs(5) == [0, 1, 0, 1, 0]
    assert m.stats() == (5, 1, 2, 0)                # 4 free; 0 and 2 cached; no growth
    t = m.begin()
    assert m.find_cached_prefix(t, [9] * 4) == 4    # the cached prefix is still there


def test_a_rollback_grows_where_it_frees_nothing_private(make):
    m = make(4, 3, 6)
    r, toks = m.begin(), list(range(12))
    m.reserve(r, 12)
    m.publish(r, toks)                              # all three published
    assert m.truncate(r, 6) == (1, 3)               # the pool doubles
    assert m.table(r) == [0, 3] and m.stats() == (6, 2, 2, 1)
    c, _ = m.fork(r, 8)                             # shares 0 and 3
    m.reserve(r, 12)                                # 4 is private ...
    m.reserve(c, 16)                                # ... 5 is c's, and 1 is evicted for it
    assert m.table(r) == [0, 3, 4] and m.table(c) == [0, 3, 1, 5] and m.stats() == (6, 0, 1, 1)
    assert m.truncate(r, 5) == (3, 4) and m.table(r) == [0, 4]   # 2 stays cached
    assert m.stats() == (6, 0, 1, 1) and m.refs(6) == [2, 1, 0, 1, 1, 1]
