"""The rotary append and attention with sinks where offsets pass 32 bits, and on
several streams at once (GPU).  Block ids are labels: pages at the far end of a
pool of more than 2^31 elements give the bits of the same pages in a small one,
and calls that run together give the bits of calls one after another."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 32, 8, 128, 16
FAR = 140_000  # blocks of 16384 elements: 2.29e9 elements a pool
SCALES = dict(k_scale=0.02, v_scale=0.01)


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_paged_kv_gb300 as m
    return m


def _pools(dtype, n):
    if dtype == "fp8":
        return [torch.empty(n, HKV, BS * D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    t = torch.float32 if dtype == "f32" else torch.bfloat16
    return [torch.empty(n, HKV, BS, D, dtype=t, device="cuda") for _ in range(2)]


class Step:
    """Rows of some lengths appended whole (rotated), then decoded and prefilled."""

    def __init__(self, pkv, dtype, seed, lens, window=150, sinks=20):
        self.pkv, self.dtype, self.lens, self.window, self.sinks = pkv, dtype, lens, window, sinks
        g = torch.Generator(device="cuda").manual_seed(seed)
        t = torch.float32 if dtype == "f32" else torch.bfloat16
        rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(t)
        T = sum(lens)
        self.q, self.k, self.v = rnd(T, HQ, D), rnd(T, HKV, D), rnd(T, HKV, D)
        self.rope = pkv.make_rope(10000.0 ** (-np.arange(D // 2) / (D // 2)))
        self.pos = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in lens])
        self.chunk = min(lens)
        self.blocks = [-(-n // BS) for n in lens]
        self.kw = SCALES if dtype == "fp8" else {}

    def run(self, kp, vp, first):
        """The rows' pages are first, first + 1, ..; returns q, decode and chunk outputs."""
        pkv, lens = self.pkv, self.lens
        ids = np.arange(first, first + sum(self.blocks), dtype=np.int32)
        table = np.full((len(lens), max(self.blocks)), -1, np.int32)
        slots, at = [], 0
        for r, (n, b) in enumerate(zip(lens, self.blocks)):
            table[r, :b] = ids[at:at + b]
            slots.append(np.repeat(ids[at:at + b], BS)[:n].astype(np.int64) * BS + np.arange(n) % BS)
            at += b
        slots = torch.from_numpy(np.concatenate(slots).astype(np.int32)).cuda()
        table, L = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        qr = pkv.paged_kv_append_rope(kp, vp, slots, self.q, self.k, self.v, self.pos, self.rope,
                                      status=status, **self.kw)
        ends = np.cumsum(lens)
        last = torch.from_numpy(ends - 1).cuda()
        dec = pkv.paged_decode_attention(qr[last].contiguous(), kp, vp, table, L, self.window, D ** -0.5,
                                         status=status, sinks=self.sinks, **self.kw)
        C = self.chunk
        rows = torch.from_numpy(np.concatenate([np.arange(e - C, e) for e in ends])).cuda()
        cu = torch.arange(0, C * (len(lens) + 1), C, dtype=torch.int32, device="cuda")
        pre = pkv.paged_prefill_chunk_attention(qr[rows].contiguous(), cu, kp, vp, table, L, C, self.window,
                                                D ** -0.5, status=status, sinks=self.sinks, **self.kw)
        return qr, dec, pre, status


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_far_blocks_are_labels(pkv, dtype):
    s = Step(pkv, dtype, 900, [333, 70, 201])
    n = sum(s.blocks)
    near = s.run(*_pools(dtype, n), 0)
    kp, vp = _pools(dtype, FAR)
    far = s.run(kp, vp, FAR - n)
    torch.cuda.synchronize()
    assert int(near[3].item()) == 0 and int(far[3].item()) == 0
    for a, b in zip(near[:3], far[:3]):
        assert torch.isfinite(a.float()).all() and torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp8", "f32"])
def test_streams_at_once(pkv, dtype):
    steps = [Step(pkv, dtype, 910 + i, [400 + 37 * i, 65, 900 - 50 * i]) for i in range(3)]
    pools = [_pools(dtype, sum(s.blocks)) for s in steps]
    want = [s.run(*p, 0) for s, p in zip(steps, pools)]
    torch.cuda.synchronize()
    for p in pools:
        for t in p:
            t.fill_(0)
    streams = [torch.cuda.Stream() for _ in steps]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for s, p, st in zip(steps, pools, streams):
            with torch.cuda.stream(st):
                got.append(s.run(*p, 0))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert int(b[3].item()) == 0
            for x, y in zip(a[:3], b[:3]):
                assert torch.equal(x, y)
