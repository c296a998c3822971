"""Allocator fork, rollback, compaction and window expiry: the reference model
pinned by worked cases, then the library against the model on random
lifecycles; the page-copy list check and the rotary descriptor (host helpers)."""
import numpy as np
import pytest

from oracle.allocator_model import AllocatorModel, OutOfBlocks


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


# ---------------------------------------------------------------------------
# worked cases, on the model and on the library
# ---------------------------------------------------------------------------
class Lib:
    """The library's allocator with the model's names."""

    def __init__(self, pkv, *a):
        self.pkv, self.a = pkv, pkv.BlockAllocator(*a)

    def __getattr__(self, name):
        def call(*a):
            try:
                out = getattr(self.a, name)(*a)
            except self.pkv.PkvError as e:
                if e.code == self.pkv.PKV_ERR_OUT_OF_BLOCKS:
                    raise OutOfBlocks() from e
                raise
            if name == "table":
                return [int(x) for x in out]
            if name == "compact":
                return [(int(s), int(d)) for s, d in zip(*out)]
            return out
        return call

    def refs(self, n):
        return [self.a.refcount(b) for b in range(n)]


@pytest.fixture(params=["model", "library"])
def make(request, pkv):
    if request.param == "library":
        return lambda *a: Lib(pkv, *a)

    class M(AllocatorModel):
        def refs(self, n):
            return self.refcount[:n]
    return M


def test_fork_shares_full_blocks_and_owns_a_partial_one(make):
    m = make(4, 8, 8)
    r = m.begin()
    m.reserve(r, 14)                                # blocks 0 .. 3, the last holds two tokens
    c, copy = m.fork(r, 10)                         # two full blocks, two tokens of block 2
    assert m.table(c) == [0, 1, 4] and copy == (2, 4)
    assert m.refs(5) == [2, 2, 1, 1, 1]
    d, copy = m.fork(r, 8)                          # on a boundary: nothing to copy
    assert m.table(d) == [0, 1] and copy is None and m.refs(2) == [3, 3]
    e, copy = m.fork(r, 0)
    assert m.table(e) == [] and copy is None
    m.release(r)
    assert m.refs(5) == [2, 2, 0, 0, 1]
    m.release(c)
    m.release(d)
    assert m.stats()[:3] == (8, 8, 0)


def test_fork_of_a_published_prefix_publishes_no_block_twice(make):
    m = make(4, 8, 8)
    toks = list(range(9))
    r = m.begin()
    m.reserve(r, 9)
    m.publish(r, toks)
    c, copy = m.fork(r, 9)
    assert copy == (2, 3)
    m.publish(c, toks + [9, 10, 11])                # its own third block is full now
    m.release(r)
    m.release(c)
    assert m.stats()[:3] == (8, 5, 3)               # blocks 0, 1 and 3 cached
    s = m.begin()
    assert m.find_cached_prefix(s, toks + [9, 10, 11]) == 12 and m.table(s) == [0, 1, 3]


def test_truncate_frees_and_copies_on_write(make):
    m = make(4, 8, 8)
    toks = list(range(16))
    r = m.begin()
    m.reserve(r, 16)
    assert m.truncate(r, 14) is None and m.table(r) == [0, 1, 2, 3]   # private: nothing moves
    assert m.truncate(r, 10) is None and m.table(r) == [0, 1, 2]
    m.publish(r, toks[:8])                                             # blocks 0, 1
    assert m.truncate(r, 6) == (1, 3)                                  # block 1 is in the prefix table
    assert m.table(r) == [0, 3] and m.stats()[2] == 1
    c, _ = m.fork(r, 4)
    assert m.truncate(r, 3) == (0, 2) and m.table(r) == [2] and m.table(c) == [0]
    assert m.truncate(r, 0) is None and m.table(r) == []
    m.publish(c, toks[:4])                                             # still the published chain
    s = m.begin()
    assert m.find_cached_prefix(s, toks[:8]) == 8


def test_no_block_left_changes_nothing(make):
    m = make(4, 3, 3)
    r = m.begin()
    m.reserve(r, 10)
    with pytest.raises(OutOfBlocks):
        m.fork(r, 10)
    m.publish(r, list(range(8)))
    with pytest.raises(OutOfBlocks):
        m.truncate(r, 7)
    assert m.table(r) == [0, 1, 2] and m.refs(3) == [1, 1, 1]
    with pytest.raises(OutOfBlocks):
        m.compact(2)
    assert m.stats()[0] == 3


def test_compact_moves_and_evicts(make):
    m = make(1, 10, 20)
    rs = [m.begin() for _ in range(5)]
    for i, r in enumerate(rs):
        m.reserve(r, 2)                             # blocks 2i, 2i + 1
        m.publish(r, [10 * i, 10 * i + 1])
    for i in (0, 2):
        m.release(rs[i])                            # 0, 1, 4, 5 cached, in that order
    assert m.compact(7) == [(7, 0), (8, 1), (9, 4)]  # six in use, one cached block survives
    assert m.table(rs[3]) == [6, 0] and m.table(rs[4]) == [1, 4] and m.table(rs[1]) == [2, 3]
    assert m.stats()[:3] == (7, 0, 1)
    s = m.begin()
    assert m.find_cached_prefix(s, [20, 21]) == 0   # 20's block went with the eviction
    t = m.begin()
    assert m.find_cached_prefix(t, [40, 41]) == 2 and m.table(t) == [1, 4]
    m.reserve(s, 1)                                 # the last cached block is evicted
    assert m.table(s) == [5] and m.compact(7) == []


def test_expire_window_keeps_the_sinks(make):
    m = make(4, 16, 16)
    r = m.begin()
    m.reserve(r, 40)
    m.expire_window(r, 26, 5)                       # blocks 0, 1 hold the sinks; 6 holds token 26
    assert m.table(r) == [0, 1, -1, -1, -1, -1, 6, 7, 8, 9]
    m.expire_window(r, 26, 5)
    c, copy = m.fork(r, 38)
    assert m.table(c) == [0, 1, -1, -1, -1, -1, 6, 7, 8, 2] and copy == (9, 2)
    m.expire_window(r, 39, 0)
    assert m.table(r) == [-1] * 9 + [9] and m.refs(10)[0] == 1


# ---------------------------------------------------------------------------
# random lifecycles
# ---------------------------------------------------------------------------
def _invariants(m):
    held = {}
    for t in m.tables.values():
        for b in t:
            if b >= 0:
                held[b] = held.get(b, 0) + 1
    assert m.refcount == [held.get(b, 0) for b in range(m.num_blocks)]
    states = [set(m.free), set(m.lru), set(held)]
    assert sum(len(x) for x in states) == m.num_blocks
    assert set().union(*states) == set(range(m.num_blocks))
    assert set(m.lru) <= set(m.hash_of_block)


@pytest.mark.parametrize("seed", range(12))
def test_library_matches_model_on_random_lifecycles(pkv, seed):
    bs = [1, 4, 16][seed % 3]
    init, maxb = [(8, 64), (32, 32), (0, 40), (16, 200)][seed % 4]
    rng = np.random.default_rng(100 + seed)
    m, a = AllocatorModel(bs, init, maxb), Lib(pkv, bs, init, maxb)
    live = {}   # model request id -> (library request id, tokens, whether some have expired)

    def both(name, r, *args):
        """The same call on both; "out" when both ran out of blocks."""
        out = []
        for x, q in ((m, r), (a, live[r][0] if r is not None else None)):
            try:
                out.append(getattr(x, name)(*(() if r is None else (q,)), *args))
            except OutOfBlocks:
                out.append("out")
        if name == "fork" and out[0] != "out":
            assert out[1] != "out" and out[0][1] == out[1][1]
            return out
        assert out[0] == out[1], (name, out)
        return out[0]

    for step in range(400):
        op = int(rng.integers(0, 8))
        pick = list(live)[rng.integers(0, len(live))] if live else None
        if op <= 1 or pick is None:
            toks = [int(x) for x in rng.integers(0, 3, size=int(rng.integers(1, 4 * bs + 2)))]
            r, q = m.begin(), a.begin()
            live[r] = (q, toks, False)
            both("find_cached_prefix", r, toks)
            if both("reserve", r, len(toks)) == "out":
                both("release", r)
                del live[r]
            else:
                both("publish", r, toks)
        elif op == 2:
            q, toks, gone = live[pick]
            toks = toks + [int(x) for x in rng.integers(0, 3, size=int(rng.integers(1, bs + 2)))]
            if both("reserve", pick, len(toks)) != "out":
                both("publish", pick, toks)
                live[pick] = (q, toks, gone)
        elif op == 3:
            q, toks, gone = live[pick]
            n = int(rng.integers(0, len(toks) + 1))
            f = both("fork", pick, n)
            if f != "out":
                live[f[0][0]] = (f[1][0], toks[:n], gone)
        elif op == 4:
            q, toks, gone = live[pick]
            n = int(rng.integers(0, len(toks) + 1))
            if both("truncate", pick, n) != "out":
                live[pick] = (q, toks[:n], gone)
        elif op == 5:
            both("expire_window", pick, int(rng.integers(0, len(live[pick][1]) + 1)), int(rng.integers(0, 2 * bs)))
        elif op == 6 and rng.integers(0, 3) == 0:
            both("compact", None, int(rng.integers(0, m.num_blocks + 1)))
        else:
            both("release", pick)
            del live[pick]
        assert a.stats() == m.stats(), step
        for r, (q, _, _) in live.items():
            assert a.table(q) == m.table(r)
        assert a.refs(m.num_blocks) == m.refcount
        _invariants(m)


def test_compact_capacity_and_bad_arguments(pkv):
    import ctypes
    a = pkv.BlockAllocator(1, 6, 6)
    x, y = a.begin(), a.begin()
    a.reserve(x, 3)
    a.reserve(y, 3)
    a.release(x)
    n, s, d = ctypes.c_int32(), (ctypes.c_int32 * 3)(), (ctypes.c_int32 * 3)()
    lib = ctypes.CDLL(pkv.LIB_PATH)
    lib.pkv_allocator_compact.argtypes = [ctypes.c_void_p, ctypes.c_int32] + [ctypes.c_void_p] * 2 + \
        [ctypes.c_int32, ctypes.c_void_p]
    assert lib.pkv_allocator_compact(a._a, 3, s, d, 2, ctypes.byref(n)) == pkv.PKV_ERR_INVALID_ARG and n.value == 3
    assert list(a.table(y)) == [3, 4, 5]
    assert lib.pkv_allocator_compact(a._a, 3, s, d, 3, ctypes.byref(n)) == pkv.PKV_OK
    assert list(zip(s, d)) == [(3, 0), (4, 1), (5, 2)] and list(a.table(y)) == [0, 1, 2]
    for bad in (lambda: a.compact(4), lambda: a.compact(-1), lambda: a.fork(y, 4), lambda: a.fork(99, 0),
                lambda: a.fork(y, -1), lambda: a.truncate(y, 4), lambda: a.truncate(99, 0),
                lambda: a.expire_window(y, 1, -1), lambda: a.expire_window(99, 0, 0)):
        with pytest.raises(pkv.PkvError) as e:
            bad()
        assert e.value.code == pkv.PKV_ERR_INVALID_ARG


# ---------------------------------------------------------------------------
# host helpers of the page copy and of the rotary append
# ---------------------------------------------------------------------------
def test_block_copies_check(pkv):
    ok = pkv.check_block_copies
    ok([0, 0, -1, 9], [1, 2, 1, -1], 10)              # a shared source, skipped pairs
    ok([3], [3], 10)
    ok([0, 1], [1, 0], 2, dst_num_blocks=2)           # other pools: only destinations count
    for src, dst, at in (([0, 1], [2, 2], 1), ([0, 1], [1, 2], 1), ([0, 2], [1, 0], 1), ([10], [0], 0),
                         ([0, 1], [1, 10], 1), ([3, 0], [3, 3], 1), ([0, 3], [3, 3], 1)):
        with pytest.raises(ValueError, match=f"pair {at} "):
            ok(src, dst, 10)
    with pytest.raises(ValueError, match="pair 1 "):
        ok([0, 1], [5, 5], 10, dst_num_blocks=6)
    with pytest.raises(ValueError):
        ok([0], [0, 1], 10)


def test_rope_descriptor_is_the_rounded_fraction_of_a_turn(pkv):
    mp = pytest.importorskip("mpmath")
    mp.mp.prec = 400
    rng = np.random.default_rng(5)
    freqs = [1.0, -1.0, 3.0, -2.5, 1e-9, 0.0, 100.25, 1e-300, -1e-19, 2.0 ** -60, 2 * np.pi, 12345678.9, -1e15]
    freqs += [float(x) for x in rng.uniform(-1, 1, 500) * 10.0 ** rng.uniform(-12, 6, 500)]
    for i in range(0, len(freqs), 128):
        part = freqs[i:i + 128]
        for f, got in zip(part, pkv.make_rope(part)._c.freq):
            want = mp.mpf(f) / (2 * mp.pi)
            off = (got - (want - mp.floor(want)) * 2 ** 64) % 2 ** 64
            # half a unit, and the double's own 2^-106 of the angle for huge frequencies
            assert min(off, 2 ** 64 - off) <= 0.5 + 1e-6 + abs(f) * 2.0 ** -40, f


def test_rope_descriptor_refusals(pkv):
    r = pkv.make_rope([1.0, 0.5], axis_of_pair=[0, 2], num_axes=3, interleaved=True, factor=2.0)
    assert r.rotary_dim == 4 and r.num_axes == 3 and r._c.axis[1] == 2 and r._c.interleaved == 1
    for bad in (lambda: pkv.make_rope([]), lambda: pkv.make_rope([float("nan")]), lambda: pkv.make_rope([1.0] * 129),
                lambda: pkv.make_rope([1.0], axis_of_pair=[4]), lambda: pkv.make_rope([1.0], axis_of_pair=[-1]),
                lambda: pkv.make_rope([1.0], axis_of_pair=[1], num_axes=1),
                lambda: pkv.make_rope([1.0], factor=float("inf")), lambda: pkv.make_rope([1.0], num_axes=0)):
        with pytest.raises(pkv.PkvError) as e:
            bad()
        assert e.value.code == pkv.PKV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        pkv.make_rope([1.0], axis_of_pair=[0, 0])
