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
