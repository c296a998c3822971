"""Latent attention over long rows (GPU), held to more than an elementwise bound: every key
is counted once, and the output's 2-norm error is that of its roundings.

Counting.  With queries of 0 every weight is 1 (exp2(0)), exactly in every type and in
every piece, so that an output is a sum of latents over the number of keys.  The row of
position p is 1 in dim p % R and 0 elsewhere: out[d] = (keys of class d) / keys.  Sums of
ones are exact in fp32, the quotient is off by some steps of it, 2^-22, and the output by
half a step of its type.  One key lost or counted twice moves its class by 1 / (its
count), and every other by 1 / keys.

2-norm.  The latents are independent N(0, 1) values and n keys have similar weights.  The
tensor-core kernel's weights are bf16, e = 2^-8 at most off each, so that the error before
the output's rounding, sum p d v less d' out with d' = sum p d, has the 2-norm of
sqrt(sum p^2 d^2) against the output's sqrt(sum p^2), at most e, and |d'| <= e sqrt(sum
p^2), of which the output's share is smaller still (sum p^2 <= 0.01 here).  A rounding is uniform
between -h and h of its binade's step, at most e relative, so that each of the two parts has at most
e / sqrt(3), both together e sqrt(2 / 3) = 0.82 e, up to the scatter of such sums over
R = 256 or more dims (some 1 / sqrt(2 R) = 4 %).  Bound: e = 2^-8.  One key of 4000 lost
is 1 / sqrt(4000) = 4 e; of 20000, 1.8 e.  fp32 (the CUDA-core kernel's weights): the
output's rounding alone, e / sqrt(3), for bf16; 2^-16 for f32 as the elementwise checks have."""
import numpy as np
import pytest
import torch

import test_gpu_latent as latent
from tree_util import HALF, as_type, attend, f64, seen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


SHAPES = [
    # kind, H, R, Dr, block size, lengths before the queries
    ("bf16", 16, 512, 64, 16, [20000, 63, 4000, 1000]),
    ("bf16", 128, 512, 64, 64, [3000, 5000]),
    ("bf16", 20, 256, 64, 32, [9000, 129, 700]),
    ("bf16", 4, 256, 64, 16, [4000] * 90),
    ("bf16", 3, 128, 32, 16, [5000, 800]),
    ("f32", 4, 64, 16, 16, [4000, 333]),
]


def form(pkv, shape, kind_of_call, seed):
    kind, H, R, Dr, bs, ctx = shape
    C = None if kind_of_call == "decode" else [(7 * i) % 40 + 1 for i in range(len(ctx))]
    if kind_of_call != "decode" and H == 128:
        C = [c % 5 + 1 for c in C]
    return latent.Case(pkv, kind, H, R, Dr, ctx, C, kind_of_call == "tree", seed=seed, bs=bs)


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}-{s[1]}-{s[2]}-{s[4]}-{len(s[5])}")
@pytest.mark.parametrize("call", ["decode", "chunk", "tree"])
def test_every_key_counts_once(pkv, shape, call):
    c = form(pkv, shape, call, 1)
    R, bs = c.R, shape[4]
    for r, L in enumerate(c.lens):
        p = np.arange(int(L))
        one = np.zeros((int(L), R + c.Dr))
        one[p, p % R] = 1
        one[:, R:] = 3                                  # (the queries are 0 there too)
        slots = torch.from_numpy(c.tables[r, p // bs].astype(np.int64) * bs + p % bs).cuda()
        c.pool.view(-1, R + c.Dr)[slots] = as_type(one, c.kind).cuda()
    c.d_q.zero_()
    out = f64(c.run(pkv))
    assert int(c.status.item()) == 0
    for r, L in enumerate(c.lens):
        a, b = c.cu[r], c.cu[r + 1]
        ok = seen(int(L), int(b - a), None if c.masks is None else c.masks[a:b])
        classes = np.stack([np.bincount(np.arange(int(L)) % R, weights=w, minlength=R) for w in ok])   # [C, R]
        want = classes / ok.sum(1, keepdims=True)
        err = np.abs(out[a:b] - want[:, None])
        assert (err <= (HALF[c.act] + 2.0 ** -22) * want[:, None]).all(), f"row {r}: {err.max()}"


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}-{s[1]}-{s[2]}-{s[4]}-{len(s[5])}")
@pytest.mark.parametrize("call", ["decode", "chunk", "tree"])
def test_norm_of_the_error(pkv, shape, call):
    c = form(pkv, shape, call, 2)
    out = f64(c.run(pkv))
    assert int(c.status.item()) == 0
    q = f64(c.q)
    some = range(0, c.H, max(1, c.H // 4))
    for r in range(0, len(c.lens), max(1, len(c.lens) // 5)):
        L, a, b = int(c.lens[r]), c.cu[r], c.cu[r + 1]
        if L < 700:
            continue
        rows = f64(c.rows[r])
        ok = seen(L, int(b - a), None if c.masks is None else c.masks[a:b])
        for h in some:
            ref, _, _ = attend(q[a:b, h], rows, rows[:, :c.R], ok, c.scale)
            rel = np.linalg.norm(out[a:b, h] - ref, axis=1) / np.linalg.norm(ref, axis=1)
            assert rel.max() <= (2.0 ** -16 if c.kind == "f32" else 2.0 ** -8), f"row {r} head {h}: {rel.max()}"


@pytest.mark.parametrize("call", ["decode", "tree"])
def test_a_key_at_every_boundary(pkv, call):
    """Keys that outweigh all others, at tiles' and pages' edges and everywhere a run of few tiles can end: each query
    looks for one of them and gets its row."""
    L, H, R, Dr = 4096, 64, 256, 64
    c = latent.Case(pkv, "bf16", H, R, Dr, [L if call == "decode" else L - 8], None if call == "decode" else [8],
                    call == "tree", seed=4)
    at = np.concatenate([np.arange(0, L - 8, 64), np.arange(63, L - 8, 64), np.arange(15, L - 8, 16), np.arange(0, L - 8, 16)])
    at = np.unique(at)
    rng = np.random.RandomState(7)
    keys = rng.randn(L, R + Dr)
    c.pool.view(-1, R + Dr)[torch.from_numpy(c.tables[0, np.arange(L) // 16].astype(np.int64) * 16 + np.arange(L) % 16).cuda()] \
        = as_type(keys, "bf16").cuda()
    keys = f64(as_type(keys, "bf16"))
    T = c.d_q.shape[0]
    for first in range(0, len(at), T * H):
        want = np.resize(at[first:first + T * H], T * H).reshape(T, H)
        # q = k: q . k = |k|^2, about 320, against some 18 N(0, 1): the others' weight is exp(-200) of them
        q = as_type(keys[want], "bf16")
        c.d_q.copy_(q)
        out = f64(c.run(pkv, scale=1.0))
        assert int(c.status.item()) == 0
        assert np.array_equal(out, keys[want][..., :R])
