"""The drill that makes the prefill's softmax warps late does make them late (GPU):
a sleep has no least length, so the tests that rely on it look at the time too."""
import pytest

import pkv_inputs as gen
from gpu_util import Dev, append

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_paged_kv_gb300 as m
    return m


@pytest.mark.parametrize("prefix,chunk", [(0, 2), (700, 60), (640, 200)])
def test_late_warps_are_late(pkv, prefix, chunk):
    w = gen.prefill_workload(seed=660, dtype="bf16", num_q_heads=16, num_kv_heads=1, head_dim=128,
                             prefix_lens=[prefix], chunk_lens=[chunk], window=0)
    d = Dev(w)
    append(pkv, d)

    def times(n):
        pkv.profile_enable([pkv.KERNEL_PREFILL])
        try:
            for _ in range(n):
                pkv.paged_prefill_chunk_attention(d.q, d.cu, d.k_pool, d.v_pool, d.tables, d.seq_lens,
                                                  chunk, 0, w.scale, max_seq_len=int(w.seq_lens.max()))
            return sorted(1e3 * t for t in pkv.profile_times(pkv.KERNEL_PREFILL))
        finally:
            pkv.profile_enable()

    times(5)
    plain = times(30)[15]
    pkv.set_wait_drill(100_000_000, pkv.DRILL_LATE_CONSUMERS)
    try:
        late = times(30)[0]
    finally:
        pkv.set_wait_drill()
    # the latest of the four warps sleeps for 32 us; a product of one tile takes about 1
    assert late > plain + 10, (late, plain)
