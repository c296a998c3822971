"""Chunked prefill whose balanced schedule has fewer tiles left than CTAs (GPU):
a few (row, kv head, query-tile pair) items more than SMs, each of a few key
tiles, so that some CTAs take no part of them and every output element must be
written all the same."""
import numpy as np
import pytest

import pkv_inputs as gen
from gpu_util import Dev, append, assert_close, oracle_pools, to_f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_paged_kv_gb300 as m
    return m


@pytest.mark.parametrize("prefix,window", [(0, 0), (100, 0), (3000, 1000), (900, 70)])
@pytest.mark.parametrize("more", [1, 2, 9])
def test_few_tiles_left(pkv, orc, prefix, window, more):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    # one kv head, two items per row of 256 queries at 8 heads: (sms + more) items, rounded up
    rows = -(-(sms + more) // 2)
    w = gen.prefill_workload(seed=600 + prefix + window, dtype="bf16", num_q_heads=8, num_kv_heads=1, head_dim=128,
                             prefix_lens=[0] * (rows - 1) + [prefix], chunk_lens=[33] * (rows - 1) + [64],
                             window=window)
    d = Dev(w)
    append(pkv, d)
    _, kp, vp = oracle_pools(orc, w)
    out = torch.full_like(d.q, float("nan"))
    pkv.paged_prefill_chunk_attention(d.q, d.cu, d.k_pool, d.v_pool, d.tables, d.seq_lens, 64, w.window, w.scale,
                                      out=out, max_seq_len=int(w.seq_lens.max()), status=d.status)
    torch.cuda.synchronize()
    assert int(d.status.item()) == 0
    ref = orc.prefill(w.q, w.cu_q_lens, kp, vp, w.dtype, w.block_tables, w.seq_lens, w.window, w.scale)
    assert_close(to_f64(out), ref, "bf16", f"prefix {prefix} window {window} rows {rows}")
