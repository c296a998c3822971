"""Drafted trees whose cu_q_lens runs past the queries (GPU): such a row is reported and
left out, nothing outside q, the masks and out is read or written, and the other
rows' results are those of the sound call."""
import numpy as np
import pytest
import torch

from test_gpu_tree import Case
from tree_util import attend, check, f64, seen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


FORMS = [
    # kind, hq, hkv, D, drafts: 16 rows, one query tile, two, chunks of 16 rows, CUDA cores
    ("bf16", 8, 8, 128, [3, 4, 2]), ("fp8", 16, 8, 128, [3, 4, 2]),
    ("bf16", 32, 8, 128, [20, 9, 30]), ("fp8", 32, 8, 128, [20, 9, 30]),
    ("bf16", 32, 8, 128, [50, 9, 64]), ("fp8", 32, 8, 128, [50, 9, 64]),
    ("bf16", 8, 8, 64, [20, 9, 30]), ("f32", 4, 2, 64, [20, 9, 30]),
]


@pytest.mark.parametrize("kind,hq,hkv,D,nodes", FORMS)
@pytest.mark.parametrize("bad", ["last", "middle", "far", "negative"])
def test_rows_past_the_queries(pkv, kind, hq, hkv, D, nodes, bad):
    c = Case(pkv, kind, hq, hkv, D, [100, 30, 700], nodes, seed=2)
    T = sum(nodes)
    # q, masks and out lie within larger buffers: the queries beyond are NaN, the masks all ones
    wide = torch.full((T + 70, hq, D), float("nan"), dtype=c.act, device="cuda")
    wide[:T] = c.args[0]
    masks = torch.full((T + 70,), -1, dtype=torch.int64, device="cuda")
    masks[:T] = c.args[2]
    out = torch.full((T + 70, hq, D), 7.0, dtype=c.act, device="cuda")
    cu = c.args[1].clone()
    if bad == "last":                   # the last row passes the end by one
        cu[3], live = T + 1, [0, 1]
    elif bad == "middle":               # the row behind it then has a negative count
        cu[2], live = T + 40, [0]
    elif bad == "far":                  # nothing is computed from these that could overflow
        cu[2], cu[3], live = 2 ** 31 - 50, 2 ** 31 - 1, [0]
    else:
        cu[0], live = -2, [1, 2]
    c.args = (wide[:T], cu, masks[:T])
    got = c.run(pkv, max_q=max(nodes) + 1 if max(nodes) < 64 else 64, out=out[:T])
    torch.cuda.synchronize()
    assert int(c.status.item()) == pkv.DEV_BAD_LEN
    first = np.concatenate([[0], np.cumsum(nodes)])
    left = torch.ones(T + 70, dtype=torch.bool, device="cuda")
    for r in live:
        s = slice(int(first[r]), int(first[r + 1]))
        left[s] = False
        ok = seen(int(c.lens[r]), nodes[r], c.masks[s])
        for h in range(0, hq, 3):
            kv = h // (hq // hkv)
            ref, mag, A = attend(f64(c.q)[s, h], c.k64[r][:, kv], c.v64[r][:, kv], ok, c.scale)
            check(got[s, h], ref, mag, A, D, kind, c.act, f"row {r} head {h}")
    assert (out[left] == 7).all()


def test_no_queries(pkv):
    c = Case(pkv, "bf16", 8, 8, 128, [40], [3])
    none = torch.empty(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    m = torch.empty(0, dtype=torch.int64, device="cuda")
    c.args = (none, torch.zeros(2, dtype=torch.int32, device="cuda"), m)
    assert c.run(pkv, max_q=3).shape == (0, 8, 128) and int(c.status.item()) == 0
