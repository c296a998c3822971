"""Latent attention called without a bound on the rows' queries (GPU): every query of a
chunk or tree is answered, with the bits of the call that gives the bound."""
import numpy as np
import pytest
import torch

from test_gpu_latent import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


@pytest.mark.parametrize("kind,H,R,Dr", [("bf16", 16, 512, 64), ("bf16", 3, 64, 16), ("f32", 4, 128, 32)])
@pytest.mark.parametrize("tree", [False, True])
def test_max_q_len_left_out(pkv, kind, H, R, Dr, tree):
    c = Case(pkv, kind, H, R, Dr, [30, 200, 0, 64, 1], [9, 1, 40, 0, 30], tree, seed=H)   # 80 queries, more than a tree holds
    out = torch.full((80, H, R), float("nan"), dtype=c.act, device="cuda")
    got = pkv.paged_latent_attention(c.d_q, c.pool, c.R, c.d_tables, c.d_lens, c.scale, cu_q_lens=c.d_cu,
                                     tree_masks=c.d_masks, out=out, status=c.status)
    assert got is out
    c.check(out)
    assert torch.equal(out, c.run(pkv))


def test_max_q_len_left_out_of_a_decode(pkv):
    c = Case(pkv, "bf16", 16, 256, 64, [33, 0, 500], seed=1)
    out = pkv.paged_latent_attention(c.d_q, c.pool, c.R, c.d_tables, c.d_lens, c.scale, status=c.status)
    c.check(out)
    assert torch.equal(out, c.run(pkv))
    with pytest.raises(ValueError):
        pkv.paged_latent_attention(c.d_q, c.pool, c.R, c.d_tables, c.d_lens, c.scale, max_q_len=2)


def test_no_queries(pkv):
    c = Case(pkv, "bf16", 16, 256, 64, [33], [2], seed=1)
    none = torch.empty(0, 16, 320, dtype=torch.bfloat16, device="cuda")
    cu = torch.from_numpy(np.zeros(2, dtype=np.int32)).cuda()
    out = pkv.paged_latent_attention(none, c.pool, c.R, c.d_tables, c.d_lens, c.scale, cu_q_lens=cu)
    assert out.shape == (0, 16, 256)
