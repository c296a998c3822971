"""Calls from several host threads at once (GPU), of shapes that want different
amounts of shared memory: each thread's stream, workspace and output are its own,
no call fails and the outputs are those of the call alone."""
import ctypes
import sys
import threading

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


def both(calls, rounds):
    """Each library call, its arguments ready, `rounds` times in a host thread of
    its own (the interpreter lock is released within a call): the codes other
    than OK."""
    codes = []

    def work(call):
        codes.extend(c for c in (call() for _ in range(rounds)) if c != 0)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    interval = sys.getswitchinterval()
    sys.setswitchinterval(1e-6)
    try:
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        sys.setswitchinterval(interval)
    torch.cuda.synchronize()
    return codes


def test_f32_decode_of_two_head_sizes(pkv):
    calls, outs, keep = [], [], []
    for d, window, sinks in ((32, 0, 0), (256, 64, 4), (32, 64, 9), (256, 0, 0)):
        w = gen.decode_workload(seed=700 + d, dtype="f32", num_q_heads=4, num_kv_heads=2, head_dim=d,
                                context_lens=[40, 100], window=window)
        dev = Dev(w)
        append(pkv, dev)
        want = pkv.paged_decode_attention(dev.q, dev.k_pool, dev.v_pool, dev.tables, dev.seq_lens, window,
                                          w.scale, max_seq_len=112, sinks=sinks)
        out = torch.empty_like(dev.q)
        ws = pkv.alloc_workspace(pkv.decode_workspace_size(2, 4, 2, d, 16, 112, window, sinks=sinks), "cuda")
        pool, stream = pkv._pool(dev.k_pool, dev.v_pool), torch.cuda.Stream()
        keep.append((dev, ws, pool, stream))
        outs.append((out, want))
        a = (dev.q.data_ptr(), 4, ctypes.byref(pool), dev.tables.data_ptr(), dev.tables.shape[1],
             dev.seq_lens.data_ptr(), 2, 112, window, sinks, w.scale, out.data_ptr(), ws.data_ptr(), ws.nbytes, None,
             stream.cuda_stream)
        calls.append(lambda a=a: pkv._lib.paged_decode_attention_sinks(*a))
    torch.cuda.synchronize()
    assert not both(calls, 10000)
    assert all(torch.equal(out, want) for out, want in outs)


def test_f32_prefill_of_two_head_sizes(pkv):
    calls, outs, keep = [], [], []
    for d in (32, 256, 32, 256):
        w = gen.prefill_workload(seed=710 + d, dtype="f32", num_q_heads=4, num_kv_heads=2, head_dim=d,
                                 prefix_lens=[20], chunk_lens=[5], window=0)
        dev = Dev(w)
        append(pkv, dev)
        want = pkv.paged_prefill_chunk_attention(dev.q, dev.cu, dev.k_pool, dev.v_pool, dev.tables,
                                                 dev.seq_lens, 5, 0, w.scale, max_seq_len=32)
        out = torch.empty_like(dev.q)
        pool, stream = pkv._pool(dev.k_pool, dev.v_pool), torch.cuda.Stream()
        keep.append((dev, pool, stream))
        outs.append((out, want))
        a = (dev.q.data_ptr(), dev.cu.data_ptr(), 4, ctypes.byref(pool), dev.tables.data_ptr(), dev.tables.shape[1],
             dev.seq_lens.data_ptr(), 1, 5, 32, 0, w.scale, out.data_ptr(), None, 0, None, stream.cuda_stream)
        calls.append(lambda a=a: pkv._lib.paged_prefill_chunk_attention(*a))
    torch.cuda.synchronize()
    assert not both(calls, 10000)
    assert all(torch.equal(out, want) for out, want in outs)
