"""Drafted trees and latent caches on the CPU: masks from parents, and refusals
before any launch."""
import numpy as np
import pytest

from tree_util import random_tree


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


def test_masks_from_parents(pkv):
    assert pkv.tree_masks_host([-1, 0, 0, 1, -1, -1, 0], [0, 5, 5, 7]).tolist() == [1, 3, 5, 11, 16, 1, 3]
    chain = pkv.tree_masks_host(np.arange(64) - 1, [0, 64])
    assert chain[63] == -1 and chain[0] == 1 and chain[62] == (1 << 63) - 1
    assert pkv.tree_masks_host([], [0, 0]).size == 0
    rng = np.random.RandomState(0)
    for _ in range(20):
        n = rng.randint(1, 65)
        up = random_tree(rng, n)
        m = pkv.tree_masks_host(up, [0, n])
        for i in range(n):
            walk, bits = i, 0
            while walk >= 0:
                bits |= 1 << int(walk)
                walk = up[walk]
            assert int(m[i]) & (1 << 64) - 1 == bits


@pytest.mark.parametrize("up,cu", [([0], [0, 1]), ([-2], [0, 1]), ([-1, 2, 0], [0, 3]), ([-1] * 65, [0, 65]),
                                   ([-1, -1, 1], [0, 1, 3])])
def test_masks_refused(pkv, up, cu):
    if up == [-1, -1, 1]:           # parent 1 of node 1: itself
        pass
    with pytest.raises(pkv.PkvError):
        pkv.tree_masks_host(up, cu)


def test_masks_arguments(pkv):
    for up, cu in (([-1], [0, 2]), ([-1], [1, 1]), ([-1, -1, -1], [0, 2, 1, 3])):
        with pytest.raises(ValueError):
            pkv.tree_masks_host(up, cu)


def test_refused_before_launch(pkv):
    import ctypes
    lib, bad = pkv._lib, pkv.PKV_ERR_INVALID_ARG
    pool = pkv._Pool(16, 16, 4, 16, 2, 128, pkv.PKV_BF16, 0.0, 0.0)
    P = ctypes.byref
    tree = lambda **k: lib.paged_tree_attention(  # noqa: E731
        k.get("q", 16), 16, k.get("m", 16), k.get("hq", 4), P(pool), 16, 8, 16, 1, k.get("mq", 4), 64, k.get("w", 0), 0.1, 16,
        k.get("ws", 256), 0, None, None)
    assert tree(mq=65) == bad and tree(m=None) == bad and tree(hq=3) == bad and tree(q=8) == bad and tree(w=-1) == bad
    assert tree(w=3) == pkv.PKV_ERR_UNSUPPORTED and tree(hq=34) == pkv.PKV_ERR_UNSUPPORTED
    assert tree() == pkv.PKV_ERR_WORKSPACE
    commit = lambda **k: lib.paged_tree_commit(  # noqa: E731
        P(k.get("pool", pool)), k.get("n", 1), 16, 8, 16, 16, 1, 16, k.get("mp", 4), 16, k.get("new", 64), None, None)
    assert commit(n=0) == bad and commit(mp=0) == bad and commit(mp=65) == bad and commit(new=16) == bad and commit(new=None) == bad
    odd = pkv._Pool(16, 16, 4, 16, 2, 12, pkv.PKV_BF16, 0.0, 0.0)
    assert commit(pool=odd) == pkv.PKV_ERR_UNSUPPORTED
    wide = pkv._Pool(16, 16, 4, 16, 1 << 26, 128, pkv.PKV_BF16, 0.0, 0.0)   # a token's rows past 16 GB
    assert commit(pool=wide) == pkv.PKV_ERR_UNSUPPORTED
    lp = pkv._LatentPool(16, 4, 16, 512, 64, pkv.PKV_BF16)
    att = lambda **k: lib.paged_latent_attention(  # noqa: E731
        16, k.get("nq", 4), k.get("cu", 16), k.get("m"), k.get("h", 4), P(k.get("pool", lp)), 16, 8, 16, 1, k.get("mq", 4), 64,
        k.get("s", 0.1), 16, 256, 0, None, None)
    assert att(cu=None) == bad and att(cu=None, mq=1) == bad and att(nq=-1) == bad and att(h=0) == bad and att(s=float("nan")) == bad and att(m=16, mq=65) == bad
    for shape in ((528, 64, pkv.PKV_BF16), (512, 72, pkv.PKV_BF16), (500, 64, pkv.PKV_BF16), (512, 64, pkv.PKV_FP8_E4M3)):
        assert att(pool=pkv._LatentPool(16, 4, 16, *shape)) == pkv.PKV_ERR_UNSUPPORTED
    assert att() == pkv.PKV_ERR_WORKSPACE
    assert lib.paged_tree_workspace_size(1, 4, 2, 128, 16, 65, 64, 0) == 0
    assert lib.paged_latent_workspace_size(1, 0, 512, 64, 16, 1, 64) == 0
