"""Drafted trees over the paged K/V cache: attention against a 64-bit form, the
commit of accepted paths byte for byte, their refusals and odd calls."""
import numpy as np
import pytest
import torch

from tree_util import as_type, attend, check, f64, fill, random_tree, seen, tables_for

pytestmark = pytest.mark.gpu

KS, VS = 0.0123, 0.0171


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


class Case:
    """Rows of `ctx` cached tokens and trees of `nodes` drafts; unused slots hold NaN."""

    def __init__(self, pkv, kind, hq, hkv, D, ctx, nodes, window=0, seed=0, bs=16, masks=None):
        rng = np.random.RandomState(seed)
        self.kind, self.hq, self.hkv, self.D, self.window = kind, hq, hkv, D, window
        self.act = torch.float32 if kind == "f32" else torch.bfloat16
        self.n = np.array(ctx)
        self.C = np.array(nodes)
        self.lens = self.n + self.C
        self.cu = np.concatenate([[0], np.cumsum(self.C)]).astype(np.int32)
        parents = np.concatenate([random_tree(rng, c) for c in nodes] or [[]]).astype(np.int32)
        self.masks = pkv.tree_masks_host(parents, self.cu) if masks is None else np.asarray(masks, dtype=np.int64)
        lo = np.maximum(0, self.n - window + 1) if window else None
        self.tables, nb = tables_for(rng, self.lens, lo, bs=bs)
        T = int(self.cu[-1])
        self.q = as_type(rng.randn(T, hq, D), kind)
        self.k = [as_type(rng.randn(int(L), hkv, D), kind) for L in self.lens]
        self.v = [as_type(rng.randn(int(L), hkv, D), kind) for L in self.lens]
        dev = "cuda"
        if kind == "fp8":
            self.kp, self.vp = pkv.fp8_pools(nb, hkv, D, dev)
            self.kp.fill_(0x7F)
            self.vp.fill_(0x7F)
            for r, L in enumerate(self.lens):
                pos = np.array([p for p in range(int(L)) if self.tables[r, p // bs] >= 0])
                slots = self.tables[r, pos // bs] * bs + pos % bs
                pkv.paged_kv_append(self.kp, self.vp, torch.from_numpy(slots.astype(np.int32)).to(dev),
                                    self.k[r][pos].to(dev), self.v[r][pos].to(dev), k_scale=KS, v_scale=VS)
            q8 = lambda t, s: f64((t.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn)) * s  # noqa: E731
            self.k64, self.v64 = [q8(t, KS) for t in self.k], [q8(t, VS) for t in self.v]
        else:
            kp = torch.full((nb, bs, hkv, D), float("nan"), dtype=self.act)
            vp = kp.clone()
            for r, L in enumerate(self.lens):
                fill(kp, self.tables, r, int(L), self.k[r], bs)
                fill(vp, self.tables, r, int(L), self.v[r], bs)
            self.kp, self.vp = [t.permute(0, 2, 1, 3).contiguous().to(dev) for t in (kp, vp)]
            self.k64, self.v64 = [f64(t) for t in self.k], [f64(t) for t in self.v]
        self.scale = D ** -0.5
        to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)  # noqa: E731
        self.args = (self.q.to(dev), to(self.cu), to(self.masks))
        self.d_tables, self.d_lens = to(self.tables), to(self.lens.astype(np.int32))
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)

    def run(self, pkv, max_q=None, **kw):
        return pkv.paged_tree_attention(*self.args, self.kp, self.vp, self.d_tables, self.d_lens,
                                        max_q if max_q is not None else int(self.C.max()), self.window,
                                        kw.pop("scale", self.scale), status=self.status, k_scale=KS, v_scale=VS, **kw)

    def check(self, out, scale=None):
        assert int(self.status.item()) == 0
        q = f64(self.q)
        G = self.hq // self.hkv
        for r, L in enumerate(self.lens):
            a, b = self.cu[r], self.cu[r + 1]
            ok = seen(int(L), int(b - a), self.masks[a:b], self.window)
            for h in range(self.hq):
                ref, mag, A = attend(q[a:b, h], self.k64[r][:, h // G], self.v64[r][:, h // G], ok,
                                     self.scale if scale is None else scale)
                check(out[a:b, h], ref, mag, A, self.D, self.kind, self.act, f"row {r} head {h}")


CASES = [
    # kind, hq, hkv, D, cached, drafts, window
    ("bf16", 16, 8, 128, [600], [4], 0),
    ("bf16", 16, 8, 128, [0, 1, 15, 16, 17], [1, 2, 8, 1, 3], 0),
    ("bf16", 32, 8, 128, [100, 1000, 0, 63], [16, 64, 64, 1], 0),
    ("bf16", 32, 8, 128, [2000, 5, 700], [40, 33, 64], 64),
    ("bf16", 16, 1, 128, [300, 64], [64, 5], 0),
    ("bf16", 8, 8, 64, [50, 500], [64, 17], 0),
    ("bf16", 8, 2, 64, [50, 500], [4, 3], 40),
    ("bf16", 8, 1, 256, [129, 40], [2, 7], 0),
    ("bf16", 8, 1, 256, [900], [64], 100),
    ("bf16", 6, 2, 64, [77], [20], 0),
    ("bf16", 6, 2, 128, [77, 300], [20, 64], 0),
    ("fp8", 12, 4, 128, [77, 300], [5, 31], 70),
    ("fp8", 16, 4, 128, [100, 1500, 0], [4, 2, 3], 0),
    ("fp8", 16, 4, 128, [100, 1500, 0], [64, 1, 30], 0),
    ("fp8", 16, 4, 128, [5000, 900], [30, 64], 1000),
    ("fp8", 8, 1, 256, [300], [21], 0),
    ("fp8", 8, 2, 64, [300, 31], [9, 4], 33),
    ("f32", 4, 2, 64, [37, 0, 50], [5, 64, 1], 0),
    ("f32", 4, 4, 128, [200], [23], 30),
]


@pytest.mark.parametrize("kind,hq,hkv,D,ctx,nodes,window", CASES)
def test_attention(pkv, kind, hq, hkv, D, ctx, nodes, window):
    c = Case(pkv, kind, hq, hkv, D, ctx, nodes, window, seed=len(ctx) + D + hq)
    c.check(c.run(pkv))


@pytest.mark.parametrize("kind,hq,hkv,D", [("bf16", 16, 8, 128), ("bf16", 32, 8, 128), ("fp8", 32, 8, 128), ("f32", 4, 2, 64)])
def test_chain_is_the_chunk(pkv, kind, hq, hkv, D):
    """A tree without branches is the causal chunk: bit for bit where the key range is cut alike (the decode
    kernel's plan, the f32 kernel's whole range); the tensor-core kernel levels a tree's key range over the
    GPU and cuts a chunk's evenly, and each is held to the exact result."""
    nodes = [7, 1, 5] if hq == 16 else [40, 1, 13]
    chain = np.concatenate([[(1 << (i + 1)) - 1 for i in range(c)] for c in nodes])
    c = Case(pkv, kind, hq, hkv, D, [130, 40, 900], nodes, masks=chain, seed=3)
    out = c.run(pkv)
    c.check(out)
    ref = pkv.paged_prefill_chunk_attention(c.args[0], c.args[1], c.kp, c.vp, c.d_tables, c.d_lens, max(nodes), 0,
                                            c.scale, k_scale=KS, v_scale=VS)
    if kind == "f32" or max(nodes) * hq // hkv <= 16:
        assert torch.equal(out, ref)
    else:
        c.check(ref)


@pytest.mark.parametrize("hq,D,nodes", [(8, 128, 2), (32, 128, 20), (8, 64, 20)])
def test_masks_as_given(pkv, hq, D, nodes):
    """Bits past the query count for nothing; a query without any key gives zeros; own bits may be missing."""
    rng = np.random.RandomState(5)
    m = np.array([rng.randint(0, 1 << 62) | (-1 << 63 if rng.rand() < 0.5 else 0) for _ in range(nodes)] * 2, dtype=np.int64)
    m[0] = 0                      # row 0 has no cached token: nothing to attend
    m[nodes] = -2                 # row 1: the cached tokens alone
    c = Case(pkv, "bf16", hq, 8, D, [0, 33], [nodes, nodes], masks=m, seed=1)
    out = c.run(pkv)
    c.check(out)
    assert (out[0] == 0).all()


def test_negative_scale(pkv):
    for hq, nodes in ((16, 4), (32, 30)):
        c = Case(pkv, "bf16", hq, 8, 128, [70], [nodes])
        c.check(c.run(pkv, scale=-0.07), scale=-0.07)


def test_padded_call_streams_and_graph(pkv):
    """Bounds above what the rows hold, a stream of its own, a captured call replayed on new inputs."""
    for hq, nodes in ((16, 4), (32, 30), (8, 30)):
        c = Case(pkv, "bf16", hq, 8, 64 if hq == 8 else 128, [300, 20], [nodes, 3], seed=2)
        ref = c.run(pkv)
        out = torch.empty_like(ref)
        ws = pkv.alloc_workspace(pkv.tree_workspace_size(2, hq, 8, c.D, 16, 64, 4096), "cuda")
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.run(pkv, max_q=nodes, max_seq_len=320 + nodes, workspace=ws, out=out)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                c.run(pkv, max_q=64, max_seq_len=4096, workspace=ws, out=out)
        torch.cuda.current_stream().wait_stream(s)
        c.args[0].mul_(-1)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        c.q = -c.q
        c.check(out)


def test_device_reports(pkv):
    for hq in (16, 32):
        c = Case(pkv, "bf16", hq, 8, 128, [40], [5])
        c.d_tables[0, 0] = 10000
        c.run(pkv)
        assert int(c.status.item()) == pkv.DEV_BAD_BLOCK
        c = Case(pkv, "bf16", hq, 8, 128, [0], [5])
        c.d_lens[0] = 3           # fewer tokens than drafts
        c.run(pkv)
        assert int(c.status.item()) == pkv.DEV_BAD_LEN


@pytest.mark.parametrize("kind,hq,nodes", [("bf16", 32, 20), ("bf16", 32, 50), ("fp8", 32, 20), ("fp8", 32, 50), ("bf16", 8, 2)])
def test_many_rows(pkv, kind, hq, nodes):
    """More rows than one pass of a run's plan looks at, empty ones among them; few long ones, cut many times."""
    rng = np.random.RandomState(nodes)
    B = 60
    ctx, C = rng.randint(0, 90, B), rng.randint(0, nodes + 1, B)
    ctx[3], C[5], C[6] = 1500, nodes, 0
    c = Case(pkv, kind, hq, 8, 128, ctx, C, seed=4)
    c.check(c.run(pkv))
    c = Case(pkv, kind, hq, 8, 128, [7000], [nodes], seed=5)
    c.check(c.run(pkv))


@pytest.mark.parametrize("kind,nodes", [("bf16", 2), ("bf16", 20), ("bf16", 50), ("fp8", 20), ("fp8", 50)])
def test_wait_runs_out(pkv, kind, nodes):
    """The first load withheld, the limit a millisecond: the call returns with a timeout, the next one is clean."""
    c = Case(pkv, kind, 32, 8, 128, [300, 70], [nodes, 1])
    pkv.set_wait_drill(1_000_000, pkv.DRILL_WITHHOLD_FIRST_LOAD)
    try:
        c.run(pkv)
        torch.cuda.synchronize()
    finally:
        pkv.set_wait_drill()
    assert int(c.status.item()) == pkv.DEV_TIMEOUT
    c.status.zero_()
    c.check(c.run(pkv))


@pytest.mark.parametrize("nodes", [20, 50])
def test_late_warps(pkv, nodes):
    """Softmax warps that come late to an output, over runs of several pieces."""
    c = Case(pkv, "bf16", 32, 8, 128, [700, 70, 0, 300] * 6, [nodes, 1, 7, 13] * 6)
    want = c.run(pkv)
    pkv.set_wait_drill(100_000_000, pkv.DRILL_LATE_CONSUMERS)
    try:
        got = c.run(pkv)
        torch.cuda.synchronize()
    finally:
        pkv.set_wait_drill()
    assert torch.equal(got, want)
    c.check(got)


def test_two_graphs_one_workspace(pkv):
    a, b = [Case(pkv, "bf16", 32, 8, 128, ctx, n, seed=i) for i, (ctx, n) in enumerate([([900, 40], [20, 3]), ([300], [60])])]
    ws = pkv.alloc_workspace(pkv.tree_workspace_size(2, 32, 8, 128, 16, 64, 1024), "cuda")
    want = [a.run(pkv), b.run(pkv)]
    outs = [torch.empty_like(w) for w in want]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graphs = []
        for c, o in ((a, outs[0]), (b, outs[1])):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                c.run(pkv, workspace=ws, out=o)
            graphs.append(g)
        for _ in range(3):
            for o in outs:
                o.zero_()
            for g in graphs:
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))


def test_far_pages(pkv):
    """Pages past 2^32 elements of a pool: attention and the commit."""
    nb, hkv, D, C, L = 270_000, 8, 128, 20, 100        # 4.42e9 elements, 8.8 GB a pool
    rng = np.random.RandomState(0)
    kp, vp = [torch.empty(nb, hkv, 16, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = np.concatenate([rng.choice(1000, 3, replace=False), nb - 1 - rng.choice(1000, 4, replace=False)])
    k, v = [as_type(rng.randn(L, hkv, D), "bf16") for _ in range(2)]
    for pool, x in ((kp, k), (vp, v)):
        for p in range(L):
            pool[table[p // 16], :, p % 16] = x[p].cuda()
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    t, lens, cu = to(table[None].astype(np.int32)), to(np.array([L], dtype=np.int32)), to(np.array([0, C], dtype=np.int32))
    masks = pkv.tree_masks_host(random_tree(rng, C), [0, C])
    q = as_type(rng.randn(C, 32, D), "bf16")
    out = pkv.paged_tree_attention(q.cuda(), cu, to(masks), kp, vp, t, lens, C, 0, 0.1)
    for h in range(0, 32, 7):
        ref, mag, A = attend(f64(q)[:, h], f64(k)[:, h // 4], f64(v)[:, h // 4], seen(L, C, masks), 0.1)
        check(out[:, h], ref, mag, A, D, "bf16", torch.bfloat16)
    path = np.array([[1, 4, 17]], dtype=np.int32)
    new = pkv.paged_tree_commit(pkv.PoolSet([(kp, vp)]), t, lens, cu, to(path), to(np.array([3], dtype=np.int32)))
    n = L - C
    assert new.tolist() == [n + 3]
    for pool, x in ((kp, k), (vp, v)):
        for i, a in enumerate(path[0]):
            assert torch.equal(pool[table[(n + i) // 16], :, (n + i) % 16].cpu(), x[n + a])


def test_refusals(pkv):
    c = Case(pkv, "bf16", 16, 8, 128, [40], [5])
    q, cu, m = c.args
    call = lambda **kw: pkv.paged_tree_attention(  # noqa: E731
        kw.get("q", q), kw.get("cu", cu), kw.get("m", m), c.kp, c.vp, c.d_tables, c.d_lens, kw.get("max_q", 5),
        kw.get("window", 0), 0.1, workspace=kw.get("ws"))
    with pytest.raises(pkv.PkvError) as e:
        call(max_q=65)
    assert e.value.code == pkv.PKV_ERR_INVALID_ARG
    with pytest.raises(pkv.PkvError) as e:
        call(window=4)
    assert e.value.code == pkv.PKV_ERR_UNSUPPORTED
    with pytest.raises(pkv.PkvError) as e:
        call(ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.code == pkv.PKV_ERR_WORKSPACE
    for bad in (dict(m=m.int()), dict(m=m[:-1]), dict(m=m.cpu()), dict(cu=cu[:-1]), dict(q=q.float()),
                dict(q=q.transpose(0, 1)), dict(cu=cu.long())):
        with pytest.raises(ValueError):
            call(**bad)
    assert call(max_q=5).shape == q.shape


# ---------------------------------------------------------------------------
# commit
# ---------------------------------------------------------------------------
def commit_form(kind, values, tables, lens, C, paths, bs):
    """values [nb, bs, ...] per tensor: rows moved position by position from a copy."""
    out = [v.copy() for v in values]
    for r, path in enumerate(paths):
        n = lens[r] - C[r]
        for i, a in enumerate(path):
            (sb, so), (db, do) = [(tables[r, p // bs], p % bs) for p in (n + a, n + i)]
            for v, o in zip(values, out):
                o[db, do] = v[sb, so]
    return out


def fp8_rows(pool, D, is_v):
    """[nb, hkv, 16 D] tile bytes as [nb, 16, hkv, D] codes, and the byte order."""
    t, d = np.arange(16)[:, None], np.arange(D)[None, :]
    if is_v:
        at = (d // 32) * 512 + ((d % 8) * 4 + (t % 8) // 2) * 16 + ((d % 32) // 8) * 4 + t % 2 + 2 * (t // 8)
    else:
        k = d % 16
        at = (d // 64) * 1024 + (t // 8) * 512 + ((t % 8) * 4 + (k % 8) // 2) * 16 + ((d % 64) // 16) * 4 + k % 2 + 2 * (k // 8)
    return pool[:, :, at].transpose(0, 2, 1, 3)


@pytest.mark.parametrize("kind,hkv,D,layers,bs", [
    ("bf16", 8, 128, 3, 16), ("bf16", 1, 256, 1, 16), ("f32", 2, 64, 2, 16), ("f32", 1, 32, 2, 5), ("fp8", 4, 128, 2, 16),
    ("fp8", 2, 64, 1, 16), ("fp8", 1, 256, 3, 16), ("latent", 1, 576, 2, 16), ("latent", 1, 320, 130, 32), ("bf16", 2, 64, 70, 16)])
def test_commit(pkv, kind, hkv, D, layers, bs):
    rng = np.random.RandomState(D + layers)
    n, C = np.array([0, 5, 31, 100, 7]), np.array([64, 1, 20, 64, 9])
    lens = n + C
    paths = [sorted(rng.choice(64, 40, replace=False)), [0], [], list(range(24, 64)), [0, 1, 3, 4, 8]]
    tables, nb = tables_for(rng, lens, bs=bs)
    cache = rng.randint(0, 256, (layers, 2, nb, hkv, bs, D * (1 if kind == "fp8" else 4 if kind == "f32" else 2))).astype(np.uint8)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    if kind == "latent":
        cache = cache[:, 0, :, 0]                      # [layers, nb, bs, bytes]
        dev = to(cache).view(torch.bfloat16)
        pools = pkv.LatentPoolSet(list(dev))
    elif kind == "fp8":
        dev = to(cache.reshape(layers, 2, nb, hkv, bs * D))
        pools = pkv.PoolSet([(x[0], x[1]) for x in dev])
    else:
        dev = to(cache).view(torch.float32 if kind == "f32" else torch.bfloat16)
        pools = pkv.PoolSet([(x[0], x[1]) for x in dev])
    path = np.full((5, 64), -7, dtype=np.int32)
    for r, x in enumerate(paths):
        path[r, :len(x)] = x
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = pkv.paged_tree_commit(pools, to(tables), to(lens.astype(np.int32)), to(np.concatenate([[0], np.cumsum(C)]).astype(np.int32)),
                                to(path), to(np.array([len(x) for x in paths], dtype=np.int32)), status=status)
    got = dev.cpu().view(torch.uint8).numpy().reshape(cache.shape)
    assert int(status.item()) == 0
    assert new.tolist() == [int(a) + len(x) for a, x in zip(n, paths)]
    for layer in range(layers):
        for side in range(1 if kind == "latent" else 2):
            a, b = (cache[layer], got[layer]) if kind == "latent" else (cache[layer, side], got[layer, side])
            if kind == "fp8":
                a, b = [fp8_rows(x.reshape(nb, hkv, bs * D), D, side == 1) for x in (a, b)]
            elif kind != "latent":
                a, b = a.transpose(0, 2, 1, 3), b.transpose(0, 2, 1, 3)
            ref = commit_form(kind, [a], tables, lens, C, paths, bs)[0]
            assert np.array_equal(ref, b), (layer, side)


def test_commit_reports(pkv):
    """Paths that break the rules leave their row alone; missing pages skip their tokens."""
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    lens, cu = [20, 20, 20, 20, 20, 30], [0, 8, 16, 24, 32, 40, 48]
    tables = np.arange(12).reshape(6, 2)
    path = np.array([[0, 2, 2, 0], [1, 9, 0, 0], [2, 1, 0, 0], [-1, 3, 0, 0], [1, 3, 4, 0], [7, 0, 0, 0]])
    counts = [3, 2, 2, 2, 5, 1]
    pool = torch.randn(12, 2, 16, 64, device="cuda").bfloat16()
    k, v = pool.clone(), pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = pkv.paged_tree_commit(pkv.PoolSet([(k, v)]), to(tables), to(lens), to(cu), to(path), to(counts), status=status)
    assert int(status.item()) == pkv.DEV_BAD_PATH
    assert new.tolist() == [12, 12, 12, 12, 12, 23]
    want = pool.clone()
    want[11, :, 6] = pool[11, :, 13]                  # row 5: position 29 to 22
    assert torch.equal(k, want) and torch.equal(v, want)
    status.zero_()
    tables[5, 1] = 40
    new = pkv.paged_tree_commit(pkv.PoolSet([(k, v)]), to(tables), to(lens), to(cu), to(path), to([0] * 5 + [1]), status=status)
    assert int(status.item()) == pkv.DEV_BAD_BLOCK and new.tolist() == [12] * 5 + [23] and torch.equal(k, want)
    status.zero_()
    new = pkv.paged_tree_commit(pkv.PoolSet([(k, v)]), to(tables), to([40, 3, -1, 20, 20, 30]), to(cu), to(path), to([1] * 6), status=status)
    assert int(status.item()) & pkv.DEV_BAD_LEN


def test_commit_of_very_many_rows(pkv):
    """More rows than a grid's second dimension has."""
    B = 66_000
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = [torch.randn(B, 1, 16, 64, generator=g, device="cuda").bfloat16() for _ in range(2)]
    want = [x.clone() for x in (k, v)]
    i32 = dict(dtype=torch.int32, device="cuda")
    rows = torch.arange(B, **i32)
    move = torch.randint(0, 8, (B,), generator=g, device="cuda")       # draft of 8 accepted, behind 5 tokens
    tables = rows.flip(0)[:, None].contiguous()
    new = pkv.paged_tree_commit(pkv.PoolSet([(k, v)]), tables, torch.full((B,), 13, **i32), torch.arange(B + 1, **i32) * 8,
                                move[:, None].int().contiguous(), torch.ones(B, **i32))
    assert (new == 6).all()
    for x, w in zip((k, v), want):
        page = tables[:, 0].long()
        w[page, :, 5] = w[page, :, 5 + move]
        assert torch.equal(x, w)


def test_commit_refusals(pkv):
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    pool = torch.zeros(4, 2, 16, 64, device="cuda").bfloat16()
    pools = pkv.PoolSet([(pool, pool.clone())])
    lens, cu, tables, path, n = to([20]), to([0, 8]), to([[0, 1]]), to([[0, 1]]), to([2])
    with pytest.raises(pkv.PkvError):
        pkv.paged_tree_commit(pools, tables, lens, cu, path, n, new_seq_lens=lens)
    with pytest.raises(pkv.PkvError):
        pkv.paged_tree_commit(pools, tables, lens, cu, to([[0] * 65]), n)
    for bad in (dict(path=path[0]), dict(lens=lens.long()), dict(cu=cu[:1]), dict(n=n.cpu())):
        with pytest.raises(ValueError):
            pkv.paged_tree_commit(pools, tables, bad.get("lens", lens), bad.get("cu", cu), bad.get("path", path), bad.get("n", n))
    with pytest.raises(ValueError):
        pkv.LatentPoolSet([torch.zeros(4, 16, 576, device="cuda"), torch.zeros(4, 16, 320, device="cuda")])
