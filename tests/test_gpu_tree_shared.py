"""Rows that share the pages of a prefix (GPU): drafted trees and latent attention give the
bits of rows with pages of their own, and a commit leaves the shared pages alone."""
import numpy as np
import pytest
import torch

from tree_util import as_type, random_tree

pytestmark = pytest.mark.gpu

PREFIX = 640                                    # tokens, 40 pages


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


def to(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Rows:
    """Tables of rows with the same first PREFIX tokens: shared pages, and pages of their own."""

    def __init__(self, pkv, own, nodes, seed):
        rng = np.random.RandomState(seed)
        B, pb = len(own), PREFIX // 16
        self.C, self.n = np.array(nodes), PREFIX + np.array(own)
        self.lens = self.n + self.C
        self.cu = np.concatenate([[0], np.cumsum(self.C)]).astype(np.int32)
        self.up = [random_tree(rng, c) for c in nodes]
        self.masks = pkv.tree_masks_host(np.concatenate(self.up), self.cu)
        pages = -(-self.lens // 16)
        self.nb = pb + B * int(pages.max())
        ids = rng.permutation(self.nb)
        self.shared = np.full((B, int(pages.max())), -1, dtype=np.int32)
        self.private = self.shared.copy()
        self.copies = []                        # (private page, shared page)
        at = pb
        for r in range(B):
            for b in range(int(pages[r])):
                self.private[r, b] = ids[at]
                self.shared[r, b] = ids[b] if b < pb else ids[at]
                if b < pb:
                    self.copies.append((ids[at], ids[b]))
                at += 1
        self.d = [to(self.cu), to(self.masks), to(self.lens.astype(np.int32))]

    def fill(self, pool):
        a, b = np.array(self.copies).T
        pool[to(a)] = pool[to(b)]
        return pool


FORMS = [("bf16", 8, 8, 128, [3, 2, 4, 1]), ("bf16", 32, 8, 128, [16, 9, 30, 1]), ("bf16", 32, 8, 128, [64, 1, 40, 7]),
         ("fp8", 32, 8, 128, [16, 9, 30, 1]), ("fp8", 32, 8, 128, [64, 1, 40, 7]), ("bf16", 8, 2, 64, [20, 3, 9, 1]),
         ("f32", 4, 2, 64, [20, 3, 9, 1])]


@pytest.mark.parametrize("kind,hq,hkv,D,nodes", FORMS)
def test_trees(pkv, kind, hq, hkv, D, nodes):
    rows = Rows(pkv, [0, 100, 37, 900], nodes, 1)
    g = torch.Generator(device="cuda").manual_seed(3)
    act = torch.float32 if kind == "f32" else torch.bfloat16
    if kind == "fp8":
        pools = [(torch.randn(rows.nb, hkv, 16 * D, generator=g, device="cuda") / 0.02).clamp(-448, 448)
                 .to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
    else:
        pools = [torch.randn(rows.nb, hkv, 16, D, generator=g, device="cuda").to(act) for _ in range(2)]
    pools = [rows.fill(p) for p in pools]
    q = torch.randn(int(rows.cu[-1]), hq, D, generator=g, device="cuda").to(act)
    scales = dict(k_scale=0.02, v_scale=0.02) if kind == "fp8" else {}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu, masks, lens = rows.d
    out = [pkv.paged_tree_attention(q, cu, masks, *pools, to(t), lens, max(nodes), 0, D ** -0.5, status=status, **scales)
           for t in (rows.shared, rows.private)]
    assert int(status.item()) == 0 and torch.isfinite(out[0]).all()
    assert torch.equal(*out)
    # the commit: the shared pages keep their bytes, the rows' own get those of the private form
    path = np.full((4, max(nodes)), -1, dtype=np.int32)
    count = np.zeros(4, dtype=np.int32)
    for r, u in enumerate(rows.up):
        walk, node = [], len(u) - 1
        while node >= 0:
            walk, node = [node] + walk, u[node]
        path[r, :len(walk)], count[r] = walk, len(walk)
    both = []
    for t in (rows.shared, rows.private):
        mine = [p.clone() for p in pools]
        new = pkv.paged_tree_commit(pkv.PoolSet([tuple(mine)]), to(t), lens, cu, to(path), to(count), status=status)
        assert new.tolist() == (rows.n + count).tolist()
        both.append(mine)
    assert int(status.item()) == 0
    prefix = to(rows.shared[0, :PREFIX // 16]).long()
    for a, b, p in zip(*both, pools):
        assert torch.equal(a, b) and torch.equal(a[prefix], p[prefix])


@pytest.mark.parametrize("kind,H,R,Dr", [("bf16", 16, 512, 64), ("bf16", 128, 256, 64), ("f32", 4, 64, 16)])
@pytest.mark.parametrize("form", ["decode", "chunk", "tree"])
def test_latent(pkv, kind, H, R, Dr, form):
    rows = Rows(pkv, [0, 100, 37, 900], [1, 1, 1, 1] if form == "decode" else [16, 9, 30, 1], 2)
    rng = np.random.RandomState(5)
    pool = rows.fill(as_type(rng.randn(rows.nb, 16, R + Dr), kind).cuda())
    q = as_type(rng.randn(int(rows.cu[-1]), H, R + Dr) * 0.2, kind).cuda()
    cu, masks, lens = rows.d
    kw = {} if form == "decode" else dict(cu_q_lens=cu, max_q_len=30, tree_masks=masks if form == "tree" else None)
    out = [pkv.paged_latent_attention(q, pool, R, to(t), lens, 0.125, **kw) for t in (rows.shared, rows.private)]
    assert torch.isfinite(out[0]).all() and torch.equal(*out)
