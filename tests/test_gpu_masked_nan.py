"""NaN in rows that a query does not attend (GPU): in K they reach only the queries
that attend them, in every type and on every path; in f32 pools the same holds for V."""
import pytest

import pkv_inputs as gen
from gpu_util import Dev, to_torch

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_paged_kv_gb300 as m
    return m


@pytest.mark.parametrize("dtype,which", [("f32", "k"), ("f32", "v"), ("bf16", "k"), ("fp8", "k")])
@pytest.mark.parametrize("prefix,chunk", [(40, 4), (700, 60), (100, 300)])   # a verify step, key ranges, two tiles
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_a_nan_row_of_the_chunk(pkv, dtype, which, prefix, chunk, window, sinks):
    bits = "f32" if dtype == "f32" else "bf16"
    w = gen.prefill_workload(seed=950, dtype=bits, num_q_heads=8, num_kv_heads=2, head_dim=128,
                             prefix_lens=[prefix], chunk_lens=[chunk], window=window)
    d = Dev(w)
    scales = dict(k_scale=float(gen.FP8_K_SCALE), v_scale=float(gen.FP8_V_SCALE)) if dtype == "fp8" else {}
    if dtype == "fp8":
        kp, vp = pkv.fp8_pools(w.num_blocks, 2, 128, "cuda")
        slots, kr, vr = gen.live_slots(w)
        pkv.paged_kv_append(kp, vp, torch.from_numpy(slots).cuda(), to_torch(kr, "bf16"), to_torch(vr, "bf16"), **scales)
    else:
        kp, vp = d.k_pool, d.v_pool
    new = torch.from_numpy(pkv.slot_mapping_host(w.block_tables, w.num_blocks, w.new_rows, w.new_pos,
                                                 w.block_size)).cuda()
    pkv.paged_kv_append(kp, vp, new, d.k_new, d.v_new, **scales)

    def call():
        out = pkv.paged_prefill_chunk_attention(d.q, d.cu, kp, vp, d.tables, d.seq_lens, chunk, window, w.scale,
                                                max_seq_len=prefix + chunk, status=d.status, sinks=sinks, **scales)
        torch.cuda.synchronize()
        assert int(d.status.item()) == 0
        return out

    want = call()
    at = chunk // 2                                  # the chunk's row that turns NaN
    (d.k_new if which == "k" else d.v_new)[at].fill_(float("nan"))
    pkv.paged_kv_append(kp, vp, new, d.k_new, d.v_new, **scales)
    got = call()
    i = torch.arange(chunk, device="cuda")
    sees = (i >= at) & ((i - at < window) | (window == 0) | (prefix + at < sinks))
    assert torch.isnan(got[sees]).all()
    assert torch.equal(got[~sees], want[~sees])
