"""Measured cases of the operators around a drafted tree and a latent cache.

Four operators, each in a plain form (elementary torch operations) and, where
``own`` is true, as the calls a user makes of the library:

- ``tree``: the queries of a tree of drafted tokens over the paged K/V cache,
  each attending the cached tokens and its own ancestors in the tree;
- ``commit``: the accepted path's rows moved to the places right behind the
  cached tokens, in every layer's pools;
- ``latent_append``: the shared latent of each token normalised, its rotary key
  and the queries' rotary parts rotated, the row written into its page;
- ``latent``: attention whose keys and values are that one row a token
  (absorbed form): decode, chunks and drafted trees.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one stream that drafts a root and three children: latency counts
        dict(name="tree_b1_n4", op="tree", dtype="bf16", batch=1, hq=16, hkv=8, dim=128, window=0,
             ctx_min=600, ctx_max=600, nodes_min=4, nodes_max=4),
        # a serving batch, 16 drafted tokens a request
        dict(name="tree_b32_n16", op="tree", dtype="bf16", batch=32, hq=32, hkv=8, dim=128, window=0,
             ctx_min=1024, ctx_max=8192, nodes_min=16, nodes_max=16),
        # trees of unequal size over an FP8 cache's window, some of them a single token
        dict(name="tree_b16_ragged_w4096_fp8", op="tree", dtype="fp8", batch=16, hq=16, hkv=4, dim=128,
             window=4096, ctx_min=100, ctx_max=30000, nodes_min=1, nodes_max=64),
        # the accepted tokens of four requests, two layers
        dict(name="commit_b4_l2", op="commit", dtype="bf16", batch=4, hkv=8, dim=128, layers=2,
             nodes_min=8, nodes_max=8, ctx_min=100, ctx_max=2000),
        # a serving batch, every layer of a model in one call
        dict(name="commit_b64_l32", op="commit", dtype="bf16", batch=64, hkv=8, dim=128, layers=32,
             nodes_min=16, nodes_max=64, ctx_min=0, ctx_max=300),
        # a decode step of 32 requests
        dict(name="latent_append_b32", op="latent_append", dtype="bf16", tokens=32, heads=16, latent=512,
             rope=64, interleaved=True, far=131072),
        # a small model's prompt in f32, an odd length, far positions
        dict(name="latent_append_odd_777_f32", op="latent_append", dtype="f32", tokens=777, heads=4,
             latent=128, rope=32, interleaved=False, far=4000000),
        # a long context with every head
        dict(name="latent_append_16384", op="latent_append", dtype="bf16", tokens=16384, heads=128,
             latent=512, rope=64, interleaved=True, far=131072),
        # a few short streams of one rank's heads: latency counts
        dict(name="latent_decode_b4_h16", op="latent", dtype="bf16", batch=4, heads=16, latent=512, rope=64,
             tree=False, ctx_min=500, ctx_max=2000, nodes_min=1, nodes_max=1),
        # a serving batch with every head on the one GPU
        dict(name="latent_decode_b32_h128", op="latent", dtype="bf16", batch=32, heads=128, latent=512,
             rope=64, tree=False, ctx_min=1024, ctx_max=8192, nodes_min=1, nodes_max=1),
        # drafted trees over long streams
        dict(name="latent_tree_b16_h16_ragged", op="latent", dtype="bf16", batch=16, heads=16, latent=512,
             rope=64, tree=True, ctx_min=100, ctx_max=20000, nodes_min=1, nodes_max=32),
        # a prefill chunk behind a cached prefix
        dict(name="latent_chunk_2x512_h16", op="latent", dtype="bf16", batch=2, heads=16, latent=512, rope=64,
             tree=False, ctx_min=4096, ctx_max=4096, nodes_min=512, nodes_max=512),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "commit", "latent_append", "latent", "latent"])
    if op == "latent_append":
        if rng.random() < 0.2:
            return dict(op=op, dtype="f32", tokens=_log_int(rng, 1, 2000), heads=rng.choice([1, 3, 4]),
                        latent=rng.choice([128, 256]), rope=32, interleaved=rng.random() < 0.5,
                        far=_log_int(rng, 1000, 4000000))
        return dict(op=op, dtype="bf16", tokens=_log_int(rng, 1, 16384), heads=rng.choice([8, 16, 20, 64, 128]),
                    latent=rng.choice([256, 512, 512]), rope=64, interleaved=rng.random() < 0.5,
                    far=_log_int(rng, 1000, 4000000))
    nodes = _log_int(rng, 1, 64)
    lo = _log_int(rng, 1, 8000)
    base = dict(op=op, nodes_min=rng.choice([1, nodes]), nodes_max=nodes, ctx_min=rng.choice([0, lo]))
    if op == "commit":
        pool = rng.choice(["bf16", "bf16", "fp8", "latent"])
        hkv, dim = (1, 576) if pool == "latent" else rng.choice([(8, 128), (4, 128), (1, 256), (2, 64)])
        return dict(base, dtype=pool, batch=_log_int(rng, 1, 64), hkv=hkv, dim=dim,
                    layers=_log_int(rng, 1, 32), ctx_max=lo % 300 + base["ctx_min"] % 100 + 1,
                    ctx_min=base["ctx_min"] % 100)
    base["ctx_max"] = lo + _log_int(rng, 1, 8000)
    if op == "tree":
        dtype = rng.choice(["bf16", "bf16", "fp8"])
        hq, hkv, dim = rng.choice([(32, 8, 128), (16, 8, 128), (16, 4, 128), (8, 2, 64), (8, 1, 256)])
        if rng.random() < 0.15:
            dtype, hq, hkv, dim = "f32", 4, 2, 64
        if dtype != "f32" and dim != 128:      # head sizes beside 128 have their verify steps' 16 rows
            base["nodes_max"] = min(nodes, 16 * hkv // hq)
            base["nodes_min"] = min(base["nodes_min"], base["nodes_max"])
        return dict(base, dtype=dtype, batch=_log_int(rng, 1, 32), hq=hq, hkv=hkv, dim=dim,
                    window=rng.choice([0, 0, _log_int(rng, 64, 4096)]))
    if rng.random() < 0.15:
        return dict(base, dtype="f32", batch=_log_int(rng, 1, 4), heads=rng.choice([1, 3, 4]), latent=128,
                    rope=32, tree=rng.random() < 0.5, ctx_max=min(base["ctx_max"], base["ctx_min"] + 1500))
    kind = rng.choice(["decode", "tree", "chunk"])
    case = dict(base, dtype="bf16", batch=_log_int(rng, 1, 32), heads=rng.choice([8, 16, 20, 64, 128]),
                latent=rng.choice([256, 512, 512]), rope=64, tree=kind == "tree")
    if kind == "decode":
        return dict(case, nodes_min=1, nodes_max=1)
    if kind == "chunk":
        top = _log_int(rng, 2, 512)
        case.update(batch=rng.choice([1, 2]), nodes_min=rng.choice([1, top]), nodes_max=top)
    while work(case)["flops"] > 1.5e11:       # no more than the listed chunk's
        if case["ctx_max"] > 2000:
            case.update(ctx_min=case["ctx_min"] // 2, ctx_max=case["ctx_max"] // 2)
        elif case["batch"] > 2:
            case.update(batch=case["batch"] // 2)
        else:
            case.update(nodes_min=(case["nodes_min"] + 1) // 2, nodes_max=(case["nodes_max"] + 1) // 2)
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
DEV = "cuda"
K_SCALE, V_SCALE = float(np.float32(0.0123)), float(np.float32(0.0171))
_ACT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16, "latent": torch.bfloat16}


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _tile_order(dim):
    """Byte of (token, dim) in an FP8 tile, K and V: int64 [16, dim] each."""
    t = torch.arange(BLOCK, device=DEV)[:, None]
    d = torch.arange(dim, device=DEV)[None, :]
    k = d % 16
    kb = (d // 64) * 1024 + (t // 8) * 512 + ((t % 8) * 4 + (k % 8) // 2) * 16 + ((d % 64) // 16) * 4 \
        + k % 2 + 2 * (k // 8)
    vb = (d // 32) * 512 + ((d % 8) * 4 + (t % 8) // 2) * 16 + ((d % 32) // 8) * 4 + t % 2 + 2 * (t // 8)
    return kb, vb


def _pools(g, nb, hkv, dim, dtype):
    """K and V pools full of N(0, 1) values (FP8: codes of N(0, 1) / scale)."""
    if dtype != "fp8":
        return [_normal(g, (nb, hkv, BLOCK, dim), _ACT[dtype]) for _ in range(2)]
    return [(_normal(g, (nb, hkv, BLOCK * dim), torch.float32) / s).clamp(-448, 448)
            .to(torch.float8_e4m3fn).view(torch.uint8) for s in (K_SCALE, V_SCALE)]


def _inv_freq(rotary):
    return 10000.0 ** (-2.0 * np.arange(rotary // 2, dtype=np.float64) / rotary)


def _lengths(case):
    """Length (drafts counted) and drafts of each row: drawn once for a case, whatever the seed."""
    B = case["batch"]
    spread = np.random.RandomState(B * 65537 + case["ctx_max"] * 13 + case["nodes_max"])
    drafts = spread.randint(case["nodes_min"], case["nodes_max"] + 1, B)
    drafts[0] = case["nodes_max"]
    return spread.randint(case["ctx_min"], case["ctx_max"] + 1, B) + drafts, drafts


def _trees(case):
    """Every row's tree and its accepted path, drawn once for a case: ancestor masks, packed; paths."""
    rng = np.random.RandomState(case["batch"] * 31 + case["nodes_max"] * 1009)
    masks, paths = [], []
    for n in _lengths(case)[1]:
        # parents (-1: behind the last cached token), each before its children
        up = [rng.randint(-1, i) if rng.rand() < 0.6 else i - 1 for i in range(n)]
        m = []
        for i in range(n):
            m.append(1 << i | (m[up[i]] if up[i] >= 0 else 0))
        end = m[rng.randint(0, n)]
        walk = [j for j in range(n) if end >> j & 1]
        paths.append(walk[:rng.randint(0, len(walk) + 1)])
        masks += m
    return np.array(masks, dtype=np.uint64).view(np.int64), paths


def _live_tables(rng, lens, lo):
    """Block tables of rows that hold the pages from position lo on."""
    width = max(1, -(-int(lens.max()) // BLOCK))
    tables = np.full((len(lens), width), -1, dtype=np.int64)
    held = np.arange(width)[None] >= (lo // BLOCK)[:, None]
    held &= np.arange(width)[None] < -(-lens // BLOCK)[:, None]
    count = int(held.sum())
    nb = max(count, 1)
    tables[held] = rng.permutation(nb)[:count]
    return tables, nb


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 32))
    s = dict(case)
    op, act = case["op"], _ACT[case["dtype"]]
    if own:
        import block_paged_kv_gb300 as pkv
    if op == "latent_append":
        T, R, Dr, H = case["tokens"], case["latent"], case["rope"], case["heads"]
        nb = -(-T // BLOCK) + 64
        s["pool"] = _normal(g, (nb, BLOCK, R + Dr), act)
        kv = _normal(g, (T, R + Dr), act)            # one projection's output
        s["c"], s["k"] = kv[:, :R], kv[:, R:]
        s["q"] = _normal(g, (T, H, 128 + Dr), act)[..., 128:]
        s["weight"] = (1 + 0.1 * _normal(g, (R,), torch.float32)).to(act)
        if T <= 64:   # a decode step: one token per request, anywhere in its page
            slots = rng.permutation(nb)[:T] * BLOCK + rng.randint(0, BLOCK, T)
            pos = rng.randint(0, case["far"], T)
        else:         # a run of tokens through shuffled pages, starting inside one
            at = int(rng.randint(0, BLOCK)) + np.arange(T)
            slots = rng.permutation(nb)[at // BLOCK] * BLOCK + at % BLOCK
            pos = rng.randint(0, case["far"]) + np.arange(T)
        s["slots"], s["pos"] = _i32(slots), _i32(pos)
        s["blk"], s["off"] = s["slots"].long() // BLOCK, s["slots"].long() % BLOCK
        s["inv_freq"] = torch.from_numpy(_inv_freq(Dr)).to(DEV)
        # the rotated parts go behind the queries' latent parts
        s["q_out"] = torch.zeros((T, H, R + Dr), dtype=act, device=DEV)[..., R:]
        if own:
            s["desc"] = pkv.make_rope(_inv_freq(Dr), interleaved=case["interleaved"])
        return s
    lens, drafts = _lengths(case)
    masks, paths = _trees(case) if case.get("tree", True) else (None, None)
    B, n = case["batch"], lens - drafts
    s["lens"], s["cu"] = _i32(lens), _i32(np.concatenate([[0], np.cumsum(drafts)]))
    s["max_len"], s["max_q"] = int(lens.max()), int(drafts.max())
    if op == "commit":
        tables, nb = _live_tables(rng, lens, n)       # the pages of the drafts alone
        hkv, dim, layers = case["hkv"], case["dim"], case["layers"]
        if case["dtype"] == "fp8":
            shape = (layers, 2, nb, hkv, BLOCK * dim)
            s["cache"] = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
            s["k_order"], s["v_order"] = _tile_order(dim)
        elif case["dtype"] == "latent":
            s["cache"] = _normal(g, (layers, nb, BLOCK, dim), act)
        else:
            s["cache"] = _normal(g, (layers, 2, nb, hkv, BLOCK, dim), act)
        s["tables"] = _i32(tables)
        count = np.array([len(walk) for walk in paths])
        path = np.full((B, s["max_q"]), -1, dtype=np.int64)
        path[np.arange(s["max_q"])[None] < count[:, None]] = np.concatenate([*paths, []])
        s["path"], s["count"] = _i32(path), _i32(count)
        s["new_lens"] = torch.empty_like(s["lens"])
        # the same moves as pages and offsets
        row = np.repeat(np.arange(B), count)
        step = np.concatenate([np.arange(c) for c in count])
        src, dst = n[row] + path[row, step], n[row] + step
        s["src"] = [torch.from_numpy(a).to(DEV) for a in (tables[row, src // BLOCK], src % BLOCK)]
        s["dst"] = [torch.from_numpy(a).to(DEV) for a in (tables[row, dst // BLOCK], dst % BLOCK)]
        if own and case["dtype"] == "latent":
            s["pools"] = pkv.LatentPoolSet([s["cache"][i] for i in range(layers)])
        elif own:
            s["pools"] = pkv.PoolSet([(s["cache"][i, 0], s["cache"][i, 1]) for i in range(layers)])
        return s
    W = case.get("window", 0)
    tables, nb = _live_tables(rng, lens, np.maximum(0, n + 1 - W) if W else 0 * n)
    s["tables"] = _i32(tables)
    s["masks"] = torch.from_numpy(masks).to(DEV) if masks is not None else None
    total = int(drafts.sum())
    if op == "tree":
        hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
        s["k_pool"], s["v_pool"] = _pools(g, nb, hkv, dim, case["dtype"])
        s["scale"] = 1.0 / math.sqrt(dim)
        s["q"] = _normal(g, (total, hq, dim), act)
        s["out"] = torch.empty_like(s["q"])
        if case["dtype"] == "fp8":
            s["k_order"], s["v_order"] = _tile_order(dim)
        if own:
            need = pkv.tree_workspace_size(B, hq, hkv, dim, BLOCK, s["max_q"], s["max_len"], W)
    else:
        H, R, Dr = case["heads"], case["latent"], case["rope"]
        s["pool"] = _normal(g, (nb, BLOCK, R + Dr), act)
        s["scale"] = 1.0 / math.sqrt(128 + Dr)
        # absorbed queries: their products with a latent vary as those of a head of 128 dims
        s["q"] = _normal(g, (total, H, R + Dr), torch.float32)
        s["q"][..., :R] *= math.sqrt(128 / R)
        s["q"] = s["q"].to(act)
        s["out"] = torch.empty((total, H, R), dtype=act, device=DEV)
        if own:
            need = pkv.latent_workspace_size(B, H, R, Dr, BLOCK, s["max_q"], s["max_len"])
    if own:
        s["workspace"] = pkv.alloc_workspace(need, DEV)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rotate(x, cos, sin, interleaved):
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    y = (a * cos - b * sin, b * cos + a * sin)
    return torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)


def _plain_append(s):
    act = s["pool"].dtype
    angle = s["pos"].double()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    c = s["c"].float()
    c = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    k = _rotate(s["k"].float(), cos, sin, s["interleaved"])
    s["pool"][s["blk"], s["off"]] = torch.cat([c, k], -1).to(act)
    s["q_out"].copy_(_rotate(s["q"].float(), cos[:, None], sin[:, None], s["interleaved"]))
    return s["pool"], s["q_out"]


def _plain_commit(s):
    cache, (sb, so), (db, do) = s["cache"], s["src"], s["dst"]
    if s["dtype"] == "latent":
        cache[:, db, do] = cache[:, sb, so]
    elif s["dtype"] == "fp8":
        k, v, ko, vo = cache[:, 0], cache[:, 1], s["k_order"], s["v_order"]
        heads = torch.arange(s["hkv"], device=DEV)[None, :, None]
        k[:, db[:, None, None], heads, ko[do][:, None]] = k[:, sb[:, None, None], heads, ko[so][:, None]]
        v[:, db[:, None, None], heads, vo[do][:, None]] = v[:, sb[:, None, None], heads, vo[so][:, None]]
    else:
        cache.transpose(3, 4)[:, :, db, do] = cache.transpose(3, 4)[:, :, sb, so]
    torch.add(s["lens"] - (s["cu"][1:] - s["cu"][:-1]), s["count"], out=s["new_lens"])
    return cache, s["new_lens"]


def _rows(s, pool, order, scale, blk, off):
    """Pool rows at (blk, off) [B, n] as f32 [B, n, Hkv, D]."""
    if s["dtype"] != "fp8":
        return pool[blk, :, off].float()
    values = pool.view(torch.float8_e4m3fn).float() * scale
    return values[:, :, order][blk, :, off]


def _seen(s):
    """Which keys a row's queries attend: positions [n], blocks and offsets [B, n], truth values [B, C, n]."""
    C, W, cu, L = s["max_q"], s.get("window", 0), s["cu"].long(), s["lens"].long()
    at = torch.arange(C, device=DEV)
    first = (L - (cu[1:] - cu[:-1]))[:, None, None]     # position of a row's first query
    q = (cu[:-1, None] + at).clamp(max=int(s["q"].shape[0]) - 1)
    pos = torch.arange(s["max_len"], device=DEV)
    j = pos - first
    seen = (pos < L[:, None, None]) & (j <= at[:, None])
    depth = at[None].expand(len(L), C)
    if s["masks"] is not None:
        m = s["masks"][q]
        bit = (m[..., None] >> j.clamp(0, 63)) & 1
        seen = seen & ((j < 0) | (bit == 1))
        depth = ((m[..., None] >> at) & 1).sum(-1) - 1
    if W:
        seen = seen & ((j >= 0) | (pos > first + depth[..., None] - W))
    blk = s["tables"].long()[:, pos // BLOCK].clamp(min=0)
    return q, blk, (pos % BLOCK).expand_as(blk), seen


def _packed(s, o):
    """[B, C, ...] to the packed queries."""
    cu = s["cu"].long()
    i = torch.arange(s["q"].shape[0], device=DEV)
    row = torch.bucketize(i, cu[1:], right=True)
    return o[row, i - cu[row]].to(s["q"].dtype)


def _softmax(score, seen):
    score = score.masked_fill(~seen, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    return p / p.sum(-1, keepdim=True).clamp(min=1e-30)


def _plain_tree(s):
    hq, hkv, dim, B, C = s["hq"], s["hkv"], s["dim"], s["batch"], s["max_q"]
    at, blk, off, seen = _seen(s)
    k = _rows(s, s["k_pool"], s.get("k_order"), K_SCALE, blk, off)
    v = _rows(s, s["v_pool"], s.get("v_order"), V_SCALE, blk, off)
    q = s["q"][at].float().view(B, C, hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, dim)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                     # [B, Hkv, G * C, n]
    p = _softmax(score.view(B, hkv, hq // hkv, C, -1), seen[:, None, None])
    o = torch.matmul(p.view(B, hkv, -1, p.shape[-1]), v.permute(0, 2, 1, 3))
    return _packed(s, o.view(B, hq, C, dim).transpose(1, 2))


def _plain_latent(s):
    B, C, H, R = s["batch"], s["max_q"], s["heads"], s["latent"]
    at, blk, off, seen = _seen(s)
    row = s["pool"][blk, off].float()                                               # [B, n, R + Dr]
    q = s["q"][at].float().view(B, C * H, -1)
    score = (torch.matmul(q, row.transpose(1, 2)) * s["scale"]).view(B, C, H, -1)
    p = _softmax(score, seen[:, :, None])
    return _packed(s, torch.matmul(p.view(B, C * H, -1), row[..., :R]).view(B, C, H, R))


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if not own:
        return {"tree": _plain_tree, "commit": _plain_commit, "latent_append": _plain_append,
                "latent": _plain_latent}[op](s)
    import block_paged_kv_gb300 as pkv
    if op == "tree":
        return pkv.paged_tree_attention(s["q"], s["cu"], s["masks"], s["k_pool"], s["v_pool"], s["tables"],
                                        s["lens"], s["max_q"], s["window"], s["scale"], out=s["out"],
                                        workspace=s["workspace"], max_seq_len=s["max_len"],
                                        k_scale=K_SCALE, v_scale=V_SCALE)
    if op == "commit":
        pkv.paged_tree_commit(s["pools"], s["tables"], s["lens"], s["cu"], s["path"], s["count"],
                              s["new_lens"])
        return s["cache"], s["new_lens"]
    if op == "latent_append":
        pkv.paged_latent_append(s["pool"], s["slots"], s["c"], s["k"], s["pos"], s["desc"], q_rope=s["q"],
                                q_rope_out=s["q_out"], norm_weight=s["weight"], norm_eps=EPS)
        return s["pool"], s["q_out"]
    return pkv.paged_latent_attention(s["q"], s["pool"], s["latent"], s["tables"], s["lens"], s["scale"],
                                      cu_q_lens=s["cu"] if s["max_q"] > 1 else None, max_q_len=s["max_q"],
                                      tree_masks=s["masks"], out=s["out"], workspace=s["workspace"],
                                      max_seq_len=s["max_len"])


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    elem = {"f32": 4, "bf16": 2, "fp8": 1, "latent": 2}[case["dtype"]]
    act = 4 if case["dtype"] == "f32" else 2
    if op == "latent_append":
        T, R, Dr, H = case["tokens"], case["latent"], case["rope"], case["heads"]
        return {"bytes": T * (2 * (R + Dr) * act + 2 * H * Dr * act + 8) + R * act,
                "flops": T * (4 * R + 3 * (H + 1) * Dr)}
    lens, drafts = _lengths(case)
    if op == "commit":  # an accepted token that lies in its place already is not moved
        moved = sum(a != i for walk in _trees(case)[1] for i, a in enumerate(walk))
        row = case["hkv"] * case["dim"] * elem * (1 if case["dtype"] == "latent" else 2) * case["layers"]
        return {"bytes": 2 * moved * row + 4 * int(drafts.sum()) + case["batch"] * 16, "flops": 0}
    W, n = case.get("window", 0), lens - drafts
    lo = np.maximum(0, n + 1 - W) if W else 0 * n
    keys, queries = int((lens - lo).sum()), int(drafts.sum())
    pairs = int(((n - lo) * drafts).sum())
    if case.get("tree", True):
        pairs += sum(bin(m & (1 << 64) - 1).count("1") for m in _trees(case)[0].tolist())
    else:
        pairs += int((drafts * (drafts + 1) // 2).sum())
    if op == "tree":
        return {"bytes": keys * 2 * case["hkv"] * case["dim"] * elem + queries * (2 * case["hq"] * case["dim"] * act + 8)
                + keys // BLOCK * 4, "flops": 4 * case["dim"] * case["hq"] * pairs}
    H, R, Dr = case["heads"], case["latent"], case["rope"]
    return {"bytes": keys * (R + Dr) * act + queries * H * (2 * R + Dr) * act + keys // BLOCK * 4,
            "flops": 2 * H * (2 * R + Dr) * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op == "commit":
        return None  # nothing is computed
    s = prepare(case, seed)
    if op == "latent_append":
        return _exact_append(s)
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    heads = s["hq"] if op == "tree" else s["heads"]
    if sum(n * (cu[r + 1] - cu[r]) for r, n in enumerate(lens)) * heads > 1.5e9:
        return None
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    masks = s["masks"].tolist() if s["masks"] is not None else None
    for r, L in enumerate(lens):
        C = cu[r + 1] - cu[r]
        n = L - C
        allowed = np.zeros((C, L), dtype=bool)
        for i in range(C):
            mine = [j for j in range(i + 1) if masks is None or masks[cu[r] + i] >> j & 1]
            W = s.get("window", 0)
            allowed[i, max(0, n + len(mine) - W) if W else 0:n] = True
            allowed[i, [n + j for j in mine]] = True
        hidden = torch.from_numpy(~allowed).to(DEV)
        keys = torch.arange(L, device=DEV)
        blk = s["tables"][r].long()[keys // BLOCK].clamp(min=0)
        if op == "latent":
            row = s["pool"][blk, keys % BLOCK].double()
            kv = [(row, row[:, :s["latent"]])] * heads
        else:
            side = []
            for name, scale in (("k", K_SCALE), ("v", V_SCALE)):
                pool = s[name + "_pool"][blk]
                if s["dtype"] == "fp8":
                    pool = (pool.view(torch.float8_e4m3fn).double() * scale)[:, :, s[name + "_order"]]
                side.append(pool[keys, :, keys % BLOCK].double())
            G = heads // s["hkv"]
            kv = [(side[0][:, h // G], side[1][:, h // G]) for h in range(heads)]
        for h, (k, v) in enumerate(kv):
            score = s["q"][cu[r]:cu[r + 1], h].double() @ k.t() * s["scale"]
            out[cu[r]:cu[r + 1], h] = torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ v
    return out


def _exact_append(s):
    n = s["rope"] // 2
    angle = s["pos"].cpu().numpy().astype(np.longdouble)[:, None] * s["inv_freq"].cpu().numpy().astype(np.longdouble)
    turn = torch.from_numpy(np.exp(1j * np.fmod(angle, 2 * np.longdouble(np.pi)).astype(np.float64))).to(DEV)

    def rotated(x, turn):
        x = x.double()
        pair = x.unflatten(-1, (n, 2)) if s["interleaved"] else x.unflatten(-1, (2, n)).transpose(-1, -2)
        z = torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * turn
        return torch.stack([z.real, z.imag], -1 if s["interleaved"] else -2).flatten(-2)

    c = s["c"].double()
    c = c / torch.sqrt(c.square().sum(-1, keepdim=True) / s["latent"] + EPS) * s["weight"].double()
    pool = s["pool"].double()
    pool.view(-1, pool.shape[-1])[s["slots"].long()] = torch.cat([c, rotated(s["k"], turn)], -1)
    return pool, rotated(s["q"], turn[:, None])
