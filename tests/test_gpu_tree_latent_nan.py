"""NaN queries and rows in drafted trees and latent attention (GPU): a query that holds or
attends NaN gets NaN, wherever the schedule cuts its keys, and no other query changes."""
import numpy as np
import pytest
import torch

import test_gpu_latent as latent
import test_gpu_tree as tree

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


TREES = [
    # kind, hq, hkv, D, drafts: 16 rows, one query tile, two, chunks of 16 rows, CUDA cores
    ("bf16", 8, 8, 128, 4), ("fp8", 16, 8, 128, 4), ("bf16", 32, 8, 128, 20), ("fp8", 32, 8, 128, 20),
    ("bf16", 32, 8, 128, 50), ("fp8", 32, 8, 128, 50), ("bf16", 8, 8, 64, 20), ("bf16", 8, 1, 256, 5),
    ("f32", 4, 2, 64, 20),
]
CONTEXT = [[5], [70, 0, 33] * 60, [6000]]      # a tile; whole items; one item cut over the GPU


@pytest.mark.parametrize("kind,hq,hkv,D,nodes", TREES)
@pytest.mark.parametrize("ctx", CONTEXT, ids=["tile", "whole", "cut"])
def test_tree_query(pkv, kind, hq, hkv, D, nodes, ctx):
    c = tree.Case(pkv, kind, hq, hkv, D, ctx, [nodes] * len(ctx), seed=3)
    want = c.run(pkv)
    bad = [0, nodes - 1] if len(ctx) == 1 else [0, nodes + 1, nodes * len(ctx) - 1]
    c.args[0][bad] = float("nan")
    got = c.run(pkv)
    torch.cuda.synchronize()
    others = np.setdiff1d(np.arange(nodes * len(ctx)), bad)
    assert torch.isnan(got[bad]).all()
    assert torch.equal(got[others], want[others])


@pytest.mark.parametrize("kind,hq,hkv,D,nodes", TREES)
def test_tree_without_keys(pkv, kind, hq, hkv, D, nodes):
    """A NaN query that attends nothing gives zeros, as every query without a key does."""
    c = tree.Case(pkv, kind, hq, hkv, D, [0, 40], [nodes, nodes], masks=[0] * nodes + [1 << i for i in range(nodes)], seed=3)
    c.args[0][:nodes] = float("nan")
    got = c.run(pkv)
    assert (got[:nodes] == 0).all() and torch.isfinite(got).all()


@pytest.mark.parametrize("kind,hq,hkv,D,nodes", [t for t in TREES if t[0] != "fp8"])
@pytest.mark.parametrize("n", [40, 3000])
def test_tree_key(pkv, kind, hq, hkv, D, nodes, n):
    """A cached K row of NaN: every query of its row, no other row's."""
    c = tree.Case(pkv, kind, hq, hkv, D, [n, n], [nodes, nodes], seed=3)
    want = c.run(pkv)
    at = n // 2
    c.kp[c.tables[0, at // 16], :, at % 16] = float("nan")
    got = c.run(pkv)
    assert torch.isnan(got[:nodes]).all()
    assert torch.equal(got[nodes:], want[nodes:])


LATENT = [("bf16", 16, 512, 64), ("bf16", 128, 256, 64), ("bf16", 3, 128, 32), ("f32", 4, 64, 16)]


@pytest.mark.parametrize("kind,H,R,Dr", LATENT)
@pytest.mark.parametrize("ctx", CONTEXT, ids=["tile", "whole", "cut"])
@pytest.mark.parametrize("form", ["decode", "chunk", "tree"])
def test_latent_query(pkv, kind, H, R, Dr, ctx, form):
    C = None if form == "decode" else [9] * len(ctx)
    c = latent.Case(pkv, kind, H, R, Dr, [max(n, 1) for n in ctx], C, form == "tree", seed=3)
    want = c.run(pkv)
    T = want.shape[0]
    bad = sorted({0, T // 2, T - 1})
    c.d_q[bad, 1] = float("nan")                # one head of each
    got = c.run(pkv)
    torch.cuda.synchronize()
    assert torch.isnan(got[bad, 1]).all()
    keep = torch.ones(T, H, dtype=torch.bool, device="cuda")
    keep[bad, 1] = False
    assert torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("kind,H,R,Dr", LATENT)
@pytest.mark.parametrize("n", [40, 3000])
def test_latent_row(pkv, kind, H, R, Dr, n):
    c = latent.Case(pkv, kind, H, R, Dr, [n, n], seed=3)
    want = c.run(pkv)
    at = n // 2
    c.pool[c.tables[0, at // 16], at % 16] = float("nan")
    got = c.run(pkv)
    assert torch.isnan(got[0]).all()
    assert torch.equal(got[1], want[1])
