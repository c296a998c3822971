"""Latent caches: the append against the formula in 64 bits, attention over latent
rows (decode, chunks, drafted trees) against a 64-bit form, refusals and odd calls."""
import numpy as np
import pytest
import torch

from tree_util import HALF, as_type, attend, check, f64, fill, random_tree, seen, tables_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


class Case:
    def __init__(self, pkv, kind, H, R, Dr, ctx, C=None, tree=False, seed=0, bs=16):
        rng = np.random.RandomState(seed)
        self.kind, self.H, self.R, self.Dr = kind, H, R, Dr
        self.act = torch.float32 if kind == "f32" else torch.bfloat16
        self.decode = C is None
        self.C = np.array([1] * len(ctx) if C is None else C)
        self.lens = np.array(ctx) + (0 if C is None else self.C)     # decode: lengths as they are
        self.cu = np.concatenate([[0], np.cumsum(self.C)]).astype(np.int32)
        self.masks = None
        if tree:
            self.masks = pkv.tree_masks_host(np.concatenate([random_tree(rng, c) for c in self.C]), self.cu)
        self.tables, nb = tables_for(rng, self.lens, bs=bs)
        W = R + Dr
        self.rows = [as_type(rng.randn(int(L), W), kind) for L in self.lens]
        pool = torch.full((nb, bs, W), float("nan"), dtype=self.act)
        for r, L in enumerate(self.lens):
            fill(pool, self.tables, r, int(L), self.rows[r], bs)
        self.q = as_type(rng.randn(int(self.cu[-1]), H, W) * (2.0 / W) ** 0.25, kind)
        self.scale = 1.0 / np.sqrt(64)
        to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.pool, self.d_q = pool.cuda(), self.q.cuda()
        self.d_tables, self.d_lens, self.d_cu = to(self.tables), to(self.lens.astype(np.int32)), to(self.cu)
        self.d_masks = None if self.masks is None else to(self.masks)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, pkv, **kw):
        return pkv.paged_latent_attention(self.d_q, self.pool, self.R, self.d_tables, self.d_lens,
                                          kw.pop("scale", self.scale), cu_q_lens=None if self.decode else self.d_cu,
                                          max_q_len=kw.pop("max_q", int(self.C.max())), tree_masks=self.d_masks,
                                          status=self.status, **kw)

    def check(self, out, scale=None, heads=None):
        assert int(self.status.item()) == 0
        q = f64(self.q)
        for r, L in enumerate(self.lens):
            a, b = self.cu[r], self.cu[r + 1]
            rows = f64(self.rows[r])
            if L == 0:
                assert (out[a:b] == 0).all()
                continue
            ok = seen(int(L), int(b - a), None if self.masks is None else self.masks[a:b])
            for h in heads or range(self.H):
                ref, mag, A = attend(q[a:b, h], rows, rows[:, :self.R], ok, self.scale if scale is None else scale)
                check(out[a:b, h], ref, mag, A, self.R + self.Dr, "bf16 weights" if self.kind == "bf16" else self.kind, self.act, f"row {r} head {h}")


DECODE = [
    # kind, H, R, Dr, lengths, block size
    ("bf16", 16, 512, 64, [1, 16, 63, 64, 65, 1000], 16),
    ("bf16", 128, 512, 64, [700, 0, 130], 16),
    ("bf16", 20, 512, 64, [3000, 17], 16),
    ("bf16", 130, 512, 64, [90, 64], 16),
    ("bf16", 64, 256, 64, [200, 1, 4000], 16),
    ("bf16", 1, 256, 64, [33], 16),
    ("bf16", 8, 512, 64, [100, 31], 32),
    ("bf16", 8, 512, 64, [100, 200], 64),
    ("bf16", 8, 512, 64, [50, 9], 8),
    ("bf16", 3, 128, 32, [50, 9], 16),
    ("f32", 4, 128, 32, [50, 1, 0, 700], 16),
    ("f32", 17, 512, 64, [300], 7),
    ("f32", 2, 16, 16, [100], 64),
]


@pytest.mark.parametrize("kind,H,R,Dr,lens,bs", DECODE)
def test_decode(pkv, kind, H, R, Dr, lens, bs):
    c = Case(pkv, kind, H, R, Dr, lens, bs=bs, seed=H)
    c.check(c.run(pkv))


CHUNK = [
    # kind, H, R, Dr, cached, queries, tree
    ("bf16", 16, 512, 64, [0, 100, 64], [1, 40, 128], False),
    ("bf16", 128, 512, 64, [500, 3], [5, 2], False),
    ("bf16", 20, 512, 64, [70], [33], False),
    ("bf16", 16, 256, 64, [1000, 0], [70, 9], False),
    ("bf16", 16, 512, 64, [0, 100, 700], [1, 64, 30], True),
    ("bf16", 128, 512, 64, [300, 20], [3, 7], True),
    ("bf16", 8, 256, 64, [62, 126], [64, 5], True),
    ("bf16", 3, 64, 16, [62, 126], [64, 5], True),
    ("f32", 4, 128, 32, [40, 0], [17, 64], True),
    ("f32", 3, 256, 32, [40, 0], [90, 5], False),
]


@pytest.mark.parametrize("kind,H,R,Dr,ctx,C,tree", CHUNK)
def test_chunk_and_tree(pkv, kind, H, R, Dr, ctx, C, tree):
    c = Case(pkv, kind, H, R, Dr, ctx, C, tree, seed=H)
    c.check(c.run(pkv), heads=range(0, H, 1 if H < 100 else 9))


def test_many_rows(pkv):
    """More items than a pass of the run's search holds, rows of every length."""
    lens = [int(x) for x in np.random.RandomState(1).randint(0, 130, 700)]
    c = Case(pkv, "bf16", 4, 256, 64, lens, seed=9)
    c.check(c.run(pkv))
    c = Case(pkv, "f32", 2, 32, 16, lens, seed=9)
    c.check(c.run(pkv))


def test_empty_and_missing_queries(pkv):
    """Rows without a query beside others; masks that leave nothing."""
    c = Case(pkv, "bf16", 16, 512, 64, [30, 200, 0, 64], [0, 3, 2, 0], True, seed=4)
    c.masks[:] = [0, 3, 4, 0, 2]          # row 1: cached tokens; 0, 1; 2 alone.  row 2: nothing; draft 1 alone
    c.d_masks.copy_(torch.from_numpy(c.masks))
    out = c.run(pkv, max_q=3)
    c.check(out)
    assert (out[3] == 0).all()


def test_negative_and_zero_scale(pkv):
    c = Case(pkv, "bf16", 16, 512, 64, [200, 65], seed=2)
    c.check(c.run(pkv, scale=-0.05), scale=-0.05)
    c.check(c.run(pkv, scale=0.0), scale=0.0)


def test_same_call_twice_graph_and_stream(pkv):
    c = Case(pkv, "bf16", 128, 512, 64, [900, 40, 333], seed=2)
    ws = pkv.alloc_workspace(pkv.latent_workspace_size(3, 128, 512, 64, 16, 1, 4096), "cuda")
    a = c.run(pkv)
    assert torch.equal(a, c.run(pkv, workspace=ws, max_seq_len=1000))
    out = torch.empty_like(a)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(pkv, workspace=ws, out=out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run(pkv, workspace=ws, out=out)
    torch.cuda.current_stream().wait_stream(s)
    c.d_lens.copy_(torch.tensor([32, 17, 300], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    c.lens = np.array([32, 17, 300])
    c.rows = [t[:n] for t, n in zip(c.rows, c.lens)]
    c.check(out, heads=range(0, 128, 7))


def test_device_reports(pkv):
    for kind, H, R, Dr in (("bf16", 16, 512, 64), ("f32", 4, 64, 16)):
        c = Case(pkv, kind, H, R, Dr, [200])
        c.d_tables[0, 3] = -1
        out = c.run(pkv)
        assert int(c.status.item()) == pkv.DEV_BAD_BLOCK
        c.status.zero_()
        c.lens = np.array([200])
        keep = np.ones(200, dtype=bool)
        keep[48:64] = False               # the missing page counts as masked
        rows = f64(c.rows[0])
        ref, mag, A = attend(f64(c.q)[0:1, 1], rows, rows[:, :R], keep[None], c.scale)
        check(out[0:1, 1], ref, mag, A, R + Dr, "bf16 weights" if kind == "bf16" else kind, c.act)
        c = Case(pkv, kind, H, R, Dr, [100])
        c.d_lens[0] = 5000
        c.run(pkv)
        assert int(c.status.item()) & pkv.DEV_BAD_LEN
        c = Case(pkv, kind, H, R, Dr, [0], [5])
        c.d_lens[0] = 3
        c.run(pkv)
        assert int(c.status.item()) == pkv.DEV_BAD_LEN


def test_queries_bound(pkv):
    """Rows whose chunk passes the queries that the call has are reported and left out."""
    for kind, H, R, Dr in (("bf16", 16, 512, 64), ("f32", 4, 64, 16)):
        c = Case(pkv, kind, H, R, Dr, [100, 30], [3, 4])
        c.d_cu[2] = 9
        out = torch.full((7, H, R), 7.0, dtype=c.act, device="cuda")
        c.run(pkv, max_q=6, out=out)
        assert int(c.status.item()) == pkv.DEV_BAD_LEN and (out[3:] == 7).all()
        c.status.zero_()
        c.lens, c.cu = c.lens[:1], c.cu[:2]
        c.check(out[:3])


@pytest.mark.parametrize("R,C", [(512, None), (256, [40, 3])])
def test_wait_runs_out(pkv, R, C):
    """The first load withheld, the limit a millisecond: the call returns with a timeout, the next one is clean."""
    c = Case(pkv, "bf16", 16, R, 64, [300, 70], C)
    c.run(pkv)
    torch.cuda.synchronize()
    pkv.set_wait_drill(1_000_000, pkv.DRILL_WITHHOLD_FIRST_LOAD)
    try:
        c.run(pkv)
        torch.cuda.synchronize()
    finally:
        pkv.set_wait_drill()
    assert int(c.status.item()) == pkv.DEV_TIMEOUT
    c.status.zero_()
    c.check(c.run(pkv))


def test_two_graphs_one_workspace_and_calls_at_once(pkv):
    """Captured calls that share a workspace, replayed in turn; calls on two streams with one each."""
    a = Case(pkv, "bf16", 16, 512, 64, [900, 40, 333], seed=1)
    b = Case(pkv, "bf16", 16, 512, 64, [20, 500], [64, 9], True, seed=2)
    size = max(pkv.latent_workspace_size(3, 16, 512, 64, 16, 64, 1024), 1)
    ws = [pkv.alloc_workspace(size, "cuda") for _ in range(2)]
    want = [a.run(pkv), b.run(pkv)]
    outs = [torch.empty_like(w) for w in want]
    s = [torch.cuda.Stream() for _ in range(2)]
    for x in s:
        x.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s[0]):
        for c, o in ((a, outs[0]), (b, outs[1])):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s[0]):
                c.run(pkv, workspace=ws[0], out=o)
            graphs.append(g)
        for _ in range(3):
            for o in outs:
                o.zero_()
            for g in graphs:
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(s[i]):
                c.run(pkv, workspace=ws[i], out=outs[i])
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_far_pages(pkv):
    """Pages past 2^32 elements: append, decode, a tree and the commit."""
    R, Dr, H, nb = 512, 64, 16, 470_000                # 4.33e9 elements, 8.7 GB
    pool = torch.empty(nb, 16, R + Dr, dtype=torch.bfloat16, device="cuda")
    rng = np.random.RandomState(0)
    L, C = 120, 20
    table = np.concatenate([rng.choice(1000, 4, replace=False), nb - 1 - rng.choice(1000, 4, replace=False)])
    pos = np.arange(L)
    slots = torch.from_numpy((table[pos // 16] * 16 + pos % 16).astype(np.int32)).cuda()
    rope = pkv.make_rope(10000.0 ** (-2.0 * np.arange(Dr // 2) / Dr))
    c, k = [as_type(rng.randn(L, n), "bf16").cuda() for n in (R, Dr)]
    pkv.paged_latent_append(pool, slots, c, k, torch.zeros(L, dtype=torch.int32, device="cuda"), rope)
    rows = torch.cat([c, k], 1)                        # (position 0: not turned)
    assert torch.equal(pool.view(-1, R + Dr)[slots.long()], rows)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    t, lens, cu = to(table[None].astype(np.int32)), to(np.array([L], dtype=np.int32)), to(np.array([0, C], dtype=np.int32))
    masks = pkv.tree_masks_host(random_tree(rng, C), [0, C])
    q = as_type(rng.randn(C, H, R + Dr) * 0.2, "bf16")
    out = pkv.paged_latent_attention(q.cuda(), pool, R, t, lens, 0.125, cu_q_lens=cu, max_q_len=C, tree_masks=to(masks))
    one = pkv.paged_latent_attention(q[:1].cuda(), pool, R, t, lens, 0.125)
    r64 = f64(rows)
    for h in range(0, H, 5):
        ref, mag, A = attend(f64(q)[:, h], r64, r64[:, :R], seen(L, C, masks), 0.125)
        check(out[:, h], ref, mag, A, R + Dr, "bf16 weights", torch.bfloat16)
        ref, mag, A = attend(f64(q)[:1, h], r64, r64[:, :R], seen(L, 1), 0.125)
        check(one[:, h], ref, mag, A, R + Dr, "bf16 weights", torch.bfloat16)
    path = np.array([[1, 4, 17]], dtype=np.int32)
    new = pkv.paged_tree_commit(pkv.LatentPoolSet([pool]), t, lens, cu, to(path), to(np.array([3], dtype=np.int32)))
    assert new.tolist() == [L - C + 3]
    assert torch.equal(pool.view(-1, R + Dr)[slots.long()][L - C:L - C + 3], rows[[L - C + i for i in path[0]]])


def test_refusals(pkv):
    c = Case(pkv, "bf16", 16, 512, 64, [40], [5], True)
    for kw, code in ((dict(max_q=65), pkv.PKV_ERR_INVALID_ARG),
                     (dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), pkv.PKV_ERR_WORKSPACE),
                     (dict(scale=float("inf")), pkv.PKV_ERR_INVALID_ARG)):
        with pytest.raises(pkv.PkvError) as e:
            c.run(pkv, **kw)
        assert e.value.code == code
    q, pool, t, L = c.d_q, c.pool, c.d_tables, c.d_lens
    f = pkv.paged_latent_attention
    for bad in (lambda: f(q, pool, 512, t, L, 0.1), lambda: f(q.float(), pool, 512, t, L, 0.1, c.d_cu, 5),
                lambda: f(q[..., :512], pool, 512, t, L, 0.1, c.d_cu, 5), lambda: f(q, pool, 576, t, L, 0.1, c.d_cu, 5),
                lambda: f(q, pool, 512, t, L, 0.1, c.d_cu, 5, out=torch.empty_like(q)),
                lambda: f(q, pool, 512, t, L, 0.1, c.d_cu.cpu(), 5), lambda: f(q, pool, 512, t.long(), L, 0.1, c.d_cu, 5),
                lambda: f(q, pool.transpose(0, 1), 512, t, L, 0.1, c.d_cu, 5),
                lambda: f(q, pool, 512, t, L, 0.1, c.d_cu, 5, tree_masks=c.d_masks[:-1])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(pkv.PkvError) as e:
        f(torch.zeros(1, 2, 640, device="cuda").bfloat16(), torch.zeros(2, 16, 640, device="cuda").bfloat16(), 576,
          torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda"), 0.1)
    assert e.value.code == pkv.PKV_ERR_UNSUPPORTED


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
EPS = 1e-6


def rotated(x, pos, freq, interleaved):
    """x [.., T axis first .., 2n] in 64 bits by pos [T, n] positions of the pairs."""
    angle = np.fmod(pos.astype(np.longdouble) * freq.astype(np.longdouble), 2 * np.longdouble(np.pi)).astype(np.float64)
    c, s = np.cos(angle), np.sin(angle)
    while c.ndim < x.ndim:
        c, s = c[:, None], s[:, None]
    n = freq.size
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :n], x[..., n:])
    y0, y1 = a * c - b * s, b * c + a * s
    return np.stack([y0, y1], -1).reshape(x.shape) if interleaved else np.concatenate([y0, y1], -1)


@pytest.mark.parametrize("kind,T,H,R,Dr,inter,axes,norm,bs", [
    ("bf16", 1, 16, 512, 64, True, 1, True, 16), ("bf16", 33, 128, 512, 64, False, 1, True, 16),
    ("bf16", 300, 20, 256, 64, True, 1, False, 16), ("bf16", 5000, 3, 512, 64, False, 1, True, 64),
    ("bf16", 70, 5, 128, 32, True, 3, True, 16), ("bf16", 9, 1, 16, 256, False, 2, True, 16),
    ("bf16", 40, 0, 512, 64, True, 1, True, 16), ("f32", 77, 4, 128, 32, False, 1, True, 16),
    ("f32", 20, 3, 512, 8, True, 1, True, 5), ("f32", 2000, 2, 64, 128, True, 4, False, 16)])
def test_append(pkv, kind, T, H, R, Dr, inter, axes, norm, bs):
    rng = np.random.RandomState(T + H)
    act = torch.float32 if kind == "f32" else torch.bfloat16
    nb = T // bs + 9
    pool0 = as_type(rng.randn(nb, bs, R + Dr), kind)
    kv = as_type(rng.randn(T, R + Dr + 16), kind).cuda()          # rows cut from a wider projection
    c, k = kv[:, :R], kv[:, R:R + Dr]
    wide = as_type(rng.randn(T, max(H, 1), 48 + Dr), kind).cuda()
    q = wide[:, :H, 48:] if H else None
    absorbed = torch.zeros(T, max(H, 1), R + Dr, dtype=act, device="cuda")
    weight = as_type(1 + 0.3 * rng.randn(R), kind)
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    slots[T // 2] = -1 if T > 2 else slots[T // 2]
    pos = rng.randint(-2 ** 31, 2 ** 31 - 1, (axes, T)).astype(np.int32)
    freq = 10000.0 ** (-2.0 * np.arange(Dr // 2) / Dr)
    axis = np.arange(Dr // 2) % axes
    rope = pkv.make_rope(freq, axis_of_pair=axis, num_axes=axes, interleaved=inter)
    pool, status = pool0.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.paged_latent_append(pool, torch.from_numpy(slots).cuda(), c, k, torch.from_numpy(pos).cuda(), rope,
                                  q_rope=q, q_rope_out=absorbed[..., R:] if H else None,
                                  norm_weight=weight.cuda() if norm else None, norm_eps=EPS, status=status)
    assert int(status.item()) == 0
    p = pos[axis].T                                               # [T, Dr / 2]
    c64, k64 = f64(c), rotated(f64(k), p, freq, inter)
    if norm:
        c64 = c64 / np.sqrt((c64 ** 2).mean(1, keepdims=True) + EPS) * f64(weight)
    want = f64(pool0).reshape(nb * bs, R + Dr)
    live = slots >= 0
    want[slots[live]] = np.concatenate([c64, k64], 1)[live]
    got = f64(pool).reshape(want.shape)
    # half a step of the type, and fp32: the sum of R squares and three products; the
    # rotation two products of an angle exact to 2^-32 turns (its sine to 2^-23)
    assert np.array_equal(np.delete(got, slots[live], 0), np.delete(want, slots[live], 0))
    err = np.abs(got - want)
    tol_c = (HALF[act] * 1.01 + (R + 8) * 2.0 ** -24) * np.abs(want[:, :R])
    assert (err[:, :R] <= tol_c).all()
    if not norm:
        assert np.array_equal(got[slots[live]][:, :R], f64(c)[live])
    mag = 2.0 ** -21 * np.abs(f64(k)).max() + 1e-30
    assert (err[:, R:] <= HALF[act] * 1.01 * np.abs(want[:, R:]) + mag).all()
    if H:
        ref = rotated(f64(q), p, freq, inter)
        assert out.data_ptr() == absorbed[..., R:].data_ptr()
        assert (np.abs(f64(out) - ref) <= HALF[act] * 1.01 * np.abs(ref) + 2.0 ** -21 * np.abs(f64(q)).max()).all()
        assert (absorbed[..., :R] == 0).all()


def test_append_in_place_graph_and_bad_slots(pkv):
    T, H, R, Dr = 50, 16, 512, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").bfloat16()  # noqa: E731
    pool, c, k, q = torch.zeros(9, 16, R + Dr, device="cuda").bfloat16(), rnd(T, R), rnd(T, Dr), rnd(T, H, R + Dr)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.randperm(9 * 16, generator=g, device="cuda")[:T].int()
    rope = pkv.make_rope(10000.0 ** (-2.0 * np.arange(32) / 64), interleaved=True)
    ref = pkv.paged_latent_append(pool, slots, c, k, pos, rope, q_rope=q[..., R:])
    want = pool.clone()
    pool.zero_()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q2 = q.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            pkv.paged_latent_append(pool, slots, c, k, pos, rope, q_rope=q2[..., R:], q_rope_out=q2[..., R:], status=status)
    torch.cuda.current_stream().wait_stream(s)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(pool, want) and torch.equal(q2[..., R:], ref) and torch.equal(q2[..., :R], q[..., :R])
    slots[7] = 9 * 16
    graph.replay()
    torch.cuda.synchronize()
    assert int(status.item()) == pkv.DEV_BAD_SLOT


def test_append_refusals(pkv):
    T, H, R, Dr = 4, 2, 512, 64
    z = lambda *s: torch.zeros(*s, device="cuda").bfloat16()  # noqa: E731
    pool, c, k, q = z(3, 16, R + Dr), z(T, R), z(T, Dr), z(T, H, Dr)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    rope, short = [pkv.make_rope(10000.0 ** (-np.arange(n) / n)) for n in (32, 16)]
    f = pkv.paged_latent_append
    for bad in (lambda: f(pool, pos.long(), c, k, pos, rope), lambda: f(pool, pos, c[:3], k, pos, rope),
                lambda: f(pool, pos, c.float(), k, pos, rope), lambda: f(pool, pos, c, k, pos[:3], rope),
                lambda: f(pool, pos, c, k, pos, rope, q_rope=q[:3]), lambda: f(pool, pos, c, k, pos, rope, q_rope_out=q),
                lambda: f(pool, pos, c, k, pos, rope, norm_weight=z(64)), lambda: f(pool, pos, c.cpu(), k, pos, rope),
                lambda: f(pool, pos, z(R, T).t(), k, pos, rope), lambda: f(pool[:, :, :512], pos, c, k, pos, rope)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: f(pool, pos, c, k, pos, short), lambda: f(pool, pos, c, k, pos, rope, norm_weight=c[0], norm_eps=-1.0),
                lambda: f(pool, pos, z(T, R + 8)[:, 4:-4], k, pos, rope),
                lambda: f(pool, pos, c, k, pos, rope, q_rope=q, q_rope_out=q.as_strided(q.shape, (H * Dr, 0, 1)))):
        with pytest.raises(pkv.PkvError):
            bad()
