"""Chunked prefill whose bounds allow more key tiles than the balanced schedule's
32-bit sums hold (GPU): such a call takes one CTA per item, and needs no
workspace for it.  The rows themselves are short."""
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


def test_bounds_past_the_schedules_sums(pkv, orc):
    # 4 rows x 64 kv heads x 256 pairs of query tiles, 32768 key tiles each at most
    w = gen.prefill_workload(seed=650, dtype="bf16", num_q_heads=64, num_kv_heads=64, head_dim=128,
                             prefix_lens=[0, 5, 100, 30], chunk_lens=[1, 40, 3, 20], window=0)
    d = Dev(w)
    append(pkv, d)
    _, kp, vp = oracle_pools(orc, w)
    ref = orc.prefill(w.q, w.cu_q_lens, kp, vp, w.dtype, w.block_tables, w.seq_lens, 0, w.scale)
    tables = torch.full((4, 131072), -1, dtype=torch.int32, device="cuda")
    tables[:, :d.tables.shape[1]] = d.tables

    def call(max_seq_len, window, **kw):
        out = torch.full_like(d.q, float("nan"))
        pkv.paged_prefill_chunk_attention(d.q, d.cu, d.k_pool, d.v_pool, tables, d.seq_lens, 65536, window, w.scale,
                                          out=out, max_seq_len=max_seq_len, status=d.status, **kw)
        torch.cuda.synchronize()
        assert int(d.status.item()) == 0
        assert_close(to_f64(out), ref, "bf16", f"max_seq_len {max_seq_len} window {window}")

    small = pkv.alloc_workspace(256, "cuda")
    for kw in (dict(window=0), dict(window=1 << 21), dict(window=(1 << 31) - 1, sinks=(1 << 31) - 1)):
        call(1 << 21, workspace=small, **kw)            # as large a window masks nothing here
        call(1 << 21, **kw)
    # below the limit, by the lengths or by the window: the schedule, and its workspace
    for max_seq_len, window in ((1 << 20, 0), (1 << 21, 1 << 20)):
        call(max_seq_len, window)
        with pytest.raises(pkv.PkvError) as e:
            call(max_seq_len, window, workspace=small)
        assert e.value.code == pkv.PKV_ERR_WORKSPACE
