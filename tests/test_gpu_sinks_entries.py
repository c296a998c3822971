"""The C entry points with sinks, called as they are (GPU): sinks 0, or window 0
(every position visible), gives the bits of the call without sinks.  The binding
sends sinks=0 to the other entry points, so a test through it cannot tell."""
import ctypes

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


class Call:
    """A workload on the GPU, its pool as the library takes it, and a workspace."""

    def __init__(self, pkv, w, fp8):
        self.pkv, self.w, self.d = pkv, w, Dev(w)
        if fp8:
            kp, vp = pkv.fp8_pools(w.num_blocks, w.num_kv_heads, w.head_dim, "cuda")
            scales = dict(k_scale=float(gen.FP8_K_SCALE), v_scale=float(gen.FP8_V_SCALE))
            slots, kr, vr = gen.live_slots(w)
            pkv.paged_kv_append(kp, vp, torch.from_numpy(slots).cuda(), to_torch(kr, "bf16"), to_torch(vr, "bf16"),
                                **scales)
        else:
            scales = {}
            append(pkv, self.d)
            kp, vp = self.d.k_pool, self.d.v_pool
        self.kp, self.vp, self.scales = kp, vp, scales
        self.pool = pkv._pool(kp, vp, **scales)
        self.L = int(w.seq_lens.max())
        self.ws = pkv.alloc_workspace(64 << 20, "cuda")

    def decode(self, window, sinks):
        """sinks None: the entry point without them."""
        w, d, out = self.w, self.d, torch.full_like(self.d.q, float("nan"))
        a = [d.q.data_ptr(), w.num_q_heads, ctypes.byref(self.pool), d.tables.data_ptr(), d.tables.shape[1],
             d.seq_lens.data_ptr(), w.batch, self.L, window]
        b = [w.scale, out.data_ptr(), self.ws.data_ptr(), self.ws.nbytes]
        lib, st = self.pkv._lib, torch.cuda.current_stream().cuda_stream
        code = lib.paged_decode_attention(*a, *b, None, None, st) if sinks is None else \
            lib.paged_decode_attention_sinks(*a, sinks, *b, None, st)
        assert code == self.pkv.PKV_OK
        return out

    def prefill(self, window, sinks, max_q):
        w, d, out = self.w, self.d, torch.full_like(self.d.q, float("nan"))
        a = [d.q.data_ptr(), d.cu.data_ptr(), w.num_q_heads, ctypes.byref(self.pool), d.tables.data_ptr(),
             d.tables.shape[1], d.seq_lens.data_ptr(), w.batch, max_q, self.L, window]
        b = [w.scale, out.data_ptr(), self.ws.data_ptr(), self.ws.nbytes, None, torch.cuda.current_stream().cuda_stream]
        lib = self.pkv._lib
        code = lib.paged_prefill_chunk_attention(*a, *b) if sinks is None else \
            lib.paged_prefill_chunk_attention_sinks(*a, sinks, *b)
        assert code == self.pkv.PKV_OK
        return out


def same(got, want):
    return torch.equal(got, want) and not torch.isnan(want).any()


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("bf16", 128), ("bf16", 256), ("fp8", 128)])
@pytest.mark.parametrize("rows", [2, 90])
def test_decode(pkv, dtype, d, rows):
    w = gen.decode_workload(seed=900 + d, dtype="f32" if dtype == "f32" else "bf16", num_q_heads=8, num_kv_heads=2,
                            head_dim=d, context_lens=([100, 700, 0, 33] * rows)[:rows], window=0)
    c = Call(pkv, w, dtype == "fp8")
    for window, sinks in ((64, 0), (0, 0), (0, 5), (0, 2 ** 31 - 1)):
        assert same(c.decode(window, sinks), c.decode(window, None)), (window, sinks)
        lib = pkv._lib
        sizes = [8, 2, d, 16, c.L, window]
        assert lib.paged_decode_sinks_workspace_size(rows, *sizes, sinks) == \
            lib.paged_decode_workspace_size(rows, *sizes, None)
    assert not torch.equal(c.decode(64, 5), c.decode(64, None))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("hkv,prefix,chunks", [
    (2, [300, 40], [2, 3]),                                          # a verify step
    (2, [700, 90], [50, 60]),                                        # key ranges over CTAs
    (2, [640, 100], [200, 130]),
    (4, [0, 64, 500, 90, 30, 1000], [512, 300, 65, 400, 512, 512]),  # more items than SMs
])
def test_prefill(pkv, dtype, hkv, prefix, chunks):
    heads = hkv * (16 if hkv == 4 else 4)
    w = gen.prefill_workload(seed=910 + hkv, dtype="f32" if dtype == "f32" else "bf16", num_q_heads=heads,
                             num_kv_heads=hkv, head_dim=128, prefix_lens=prefix, chunk_lens=chunks, window=0)
    c = Call(pkv, w, dtype == "fp8")
    for window, sinks in ((64, 0), (0, 0), (0, 5), (0, 2 ** 31 - 1)):
        assert same(c.prefill(window, sinks, max(chunks)), c.prefill(window, None, max(chunks))), (window, sinks)
        lib = pkv._lib
        sizes = [heads, hkv, 128, 16, max(chunks), c.L, window]
        assert lib.paged_prefill_sinks_workspace_size(len(chunks), *sizes, sinks) == \
            lib.paged_prefill_workspace_size(len(chunks), *sizes)
    assert not torch.equal(c.prefill(64, 5, max(chunks)), c.prefill(64, None, max(chunks)))


def test_groups(pkv):
    c = [Call(pkv, gen.decode_workload(seed=920 + i, dtype="bf16", num_q_heads=8, num_kv_heads=1, head_dim=256,
                                       context_lens=[100, 700, 31], window=0), False) for i in range(3)]

    def run(sinks):
        outs = [torch.full_like(x.d.q, float("nan")) for x in c]
        arr = (pkv._Group * 3)()
        for g, x, out, window in zip(arr, c, outs, (0, 64, 30)):
            g.q, g.out, g.pool = x.d.q.data_ptr(), out.data_ptr(), x.pool
            g.block_tables, g.max_blocks_per_seq = x.d.tables.data_ptr(), x.d.tables.shape[1]
            g.seq_lens, g.max_seq_len, g.window, g.scale = x.d.seq_lens.data_ptr(), x.L, window, x.w.scale
        tail = [c[0].ws.data_ptr(), c[0].ws.nbytes, None, torch.cuda.current_stream().cuda_stream]
        lib = pkv._lib
        code = lib.paged_decode_attention_groups(arr, 3, 3, 8, *tail) if sinks is None else \
            lib.paged_decode_attention_groups_sinks(arr, sinks, 3, 3, 8, *tail)
        assert code == pkv.PKV_OK
        return outs

    want = run(None)
    for sinks in ((ctypes.c_int32 * 3)(0, 0, 0), (ctypes.c_int32 * 3)(7, 0, 0), 0):  # window 0 with sinks; NULL
        assert all(same(a, b) for a, b in zip(run(sinks), want))
