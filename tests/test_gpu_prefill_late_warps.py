"""Chunked prefill whose softmax warps come late to an item's output (GPU): the
tensor cores have then finished the last two products of the item, and the wait
for them must still end, for one item per CTA, key ranges cut over CTAs and the
balanced schedule's many items per CTA alike.  Being late changes no result: the
bits are those of the undisturbed call."""
import pytest

import pkv_inputs as gen
from gpu_util import Dev, append, to_torch

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_paged_kv_gb300 as m
    return m


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 0), (300, 40)])
@pytest.mark.parametrize("hkv,prefix,chunks", [
    (1, [0], [1]),              # one tile
    (1, [700], [60]),           # key ranges of one short chunk over CTAs
    (2, [640, 100], [200, 130]),
    (4, [0, 64, 500, 90, 30, 1000], [512, 300, 65, 400, 512, 512]),  # more items than SMs
])
@pytest.mark.parametrize("fp8", [False, True])
def test_late_warps_change_nothing(pkv, fp8, hkv, prefix, chunks, window, sinks):
    heads = hkv * (16 if hkv == 4 else 4)
    w = gen.prefill_workload(seed=640 + hkv, dtype="bf16", num_q_heads=heads, num_kv_heads=hkv, head_dim=128,
                             prefix_lens=prefix, chunk_lens=chunks, window=window)
    d = Dev(w)
    kw = {}
    if fp8:
        kp, vp = pkv.fp8_pools(w.num_blocks, hkv, 128, "cuda")
        kw = dict(k_scale=float(gen.FP8_K_SCALE), v_scale=float(gen.FP8_V_SCALE))
        slots, kr, vr = gen.live_slots(w)
        pkv.paged_kv_append(kp, vp, torch.from_numpy(slots).cuda(), to_torch(kr, "bf16"), to_torch(vr, "bf16"),
                            status=d.status, **kw)
    else:
        append(pkv, d)
        kp, vp = d.k_pool, d.v_pool
    if sinks:
        kw["sinks"] = sinks

    def call():
        out = torch.full_like(d.q, float("nan"))
        pkv.paged_prefill_chunk_attention(d.q, d.cu, kp, vp, d.tables, d.seq_lens, max(chunks), window, w.scale,
                                          out=out, max_seq_len=int(w.seq_lens.max()), status=d.status, **kw)
        torch.cuda.synchronize()
        assert int(d.status.item()) == 0
        return out

    want = call()
    pkv.set_wait_drill(100_000_000, pkv.DRILL_LATE_CONSUMERS)
    try:
        got = call()
    finally:
        pkv.set_wait_drill()
    assert not torch.isnan(want).any()
    assert torch.equal(got, want)
