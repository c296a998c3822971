"""The rotary append, the windowed attention with sinks and the page copies
together, as a serving loop runs them (GPU): two layers that share block ids,
requests that are prefilled in chunks, decoded, expired behind their window,
forked, rolled back and compacted.  Every step's attention is compared with
dense attention in 64 bits over the request's whole history, rotated from its
positions, which the loop keeps on the host apart from any page.

Tolerances: the framework's bf16 and f32 ones; the history holds the rotated
rows as the pool's type rounds them (bf16: from the formula in 64 bits, so a row
next to a rounding border may sit one step apart: 2^-8 relative, well inside
what the attention's own tolerance allows of one key among many).
"""
import numpy as np
import pytest

import pkv_inputs as gen
from gpu_util import assert_close, to_f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_paged_kv_gb300 as m
    return m


BS, D, HQ, HKV, LAYERS, WINDOW, SINKS = 16, 128, 8, 2, 2, 50, 5
FREQ = 10000.0 ** (-np.arange(D // 2) / (D // 2))
AXIS = np.arange(D // 2) % 3


class Loop:
    """Two layers' pools, an allocator, and every request's history on the host."""

    def __init__(self, pkv, orc, dtype, seed):
        self.pkv, self.orc, self.dtype = pkv, orc, dtype
        self.act = torch.float32 if dtype == "f32" else torch.bfloat16
        self.rng = np.random.default_rng(seed)
        self.alloc = pkv.BlockAllocator(BS, 64, 64)
        fill = float("nan")
        if dtype == "fp8":
            self.pools = [pkv.fp8_pools(64, HKV, D, "cuda") for _ in range(LAYERS)]
            for k, v in self.pools:
                k.fill_(gen.FP8_POISON)
                v.fill_(gen.FP8_POISON)
            self.sc = dict(k_scale=float(gen.FP8_K_SCALE), v_scale=float(gen.FP8_V_SCALE))
        else:
            self.pools = [tuple(torch.full((64, HKV, BS, D), fill, dtype=self.act, device="cuda") for _ in range(2))
                          for _ in range(LAYERS)]
            self.sc = {}
        self.set = pkv.PoolSet(self.pools)
        self.rope = pkv.make_rope(FREQ, AXIS)
        self.k, self.v = {}, {}        # request -> [layer] -> [n, HKV, D] float64, as the cache holds it
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def rows(self, x):
        return x.to(self.act).cuda()

    def stored(self, x, scale):
        """float64 rows as the pool's type holds them."""
        x = x.astype(np.float32)
        if self.dtype == "f32":
            return x.astype(np.float64)
        if self.dtype == "bf16":
            return gen.bf16_to_f32(gen.bf16_bits(x)).astype(np.float64)
        q = (x / np.float32(scale)).astype(np.float32)
        return self.orc.e4m3_decode(self.orc.e4m3_encode(q.reshape(-1))).reshape(x.shape) * scale

    def rotate(self, x, pos):
        th = (pos[AXIS].T * FREQ)[:, None]                 # [T, 1, D / 2]
        a, b = x[..., :D // 2], x[..., D // 2:]
        return np.concatenate([a * np.cos(th) - b * np.sin(th), b * np.cos(th) + a * np.sin(th)], -1)

    def begin(self):
        r = self.alloc.begin()
        self.k[r], self.v[r] = ([np.zeros((0, HKV, D)) for _ in range(LAYERS)] for _ in range(2))
        return r

    def copy(self, pairs):
        pairs = [p for p in pairs if p is not None]
        if pairs:
            src, dst = np.array(pairs, dtype=np.int32).T
            self.pkv.check_block_copies(src, dst, 64)
            self.pkv.paged_copy_blocks(self.set, torch.from_numpy(src.copy()).cuda(), torch.from_numpy(dst.copy()).cuda(),
                                       status=self.status)

    def step(self, counts):
        """Append counts[r] tokens to each request r of the batch and attend from them, every layer."""
        reqs = list(counts)
        before = [len(self.k[r][0]) for r in reqs]
        after = [n + counts[r] for r, n in zip(reqs, before)]
        for r, n in zip(reqs, after):
            self.alloc.reserve(r, n)
        tabs = [self.alloc.table(r) for r in reqs]
        tables = np.full((len(reqs), max(len(t) for t in tabs)), -1, dtype=np.int32)
        for i, t in enumerate(tabs):
            tables[i, :len(t)] = t
        rows = np.concatenate([np.full(counts[r], i) for i, r in enumerate(reqs)]).astype(np.int32)
        at = np.concatenate([np.arange(a, b) for a, b in zip(before, after)]).astype(np.int32)
        slots = self.pkv.slot_mapping_host(tables, 64, rows, at, BS)
        pos = np.stack([at, at // 7, at % 7]).astype(np.int32)      # time, height, width
        dev = [torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in
               (slots, pos, tables, np.array(after, dtype=np.int32), np.concatenate([[0], np.cumsum(list(counts.values()))]).astype(np.int32))]
        T = len(at)
        for layer, (kp, vp) in enumerate(self.pools):
            wide = torch.from_numpy(self.rng.standard_normal((T, (HQ + 2 * HKV) * D))).to(self.act).cuda()
            q, k, v = (wide[:, a * D:b * D].view(T, b - a, D) for a, b in ((0, HQ), (HQ, HQ + HKV), (HQ + HKV, HQ + 2 * HKV)))
            h = [x.double().cpu().numpy() for x in (q, k, v)]
            self.pkv.paged_kv_append_rope(kp, vp, dev[0], q, k, v, dev[1], self.rope, q_out=q, status=self.status, **self.sc)
            if max(counts.values()) == 1:
                out = self.pkv.paged_decode_attention(q.contiguous(), kp, vp, dev[2], dev[3], WINDOW, D ** -0.5,
                                                      status=self.status, sinks=SINKS, **self.sc)
            else:
                out = self.pkv.paged_prefill_chunk_attention(q.contiguous(), dev[4], kp, vp, dev[2], dev[3],
                                                             max(counts.values()), WINDOW, D ** -0.5,
                                                             status=self.status, sinks=SINKS, **self.sc)
            torch.cuda.synchronize()
            assert int(self.status.item()) == 0
            qr, kr = self.rotate(h[0], pos), self.rotate(h[1], pos)
            qd = to_f64(q)                # the queries the attention saw: rounded to their type
            assert np.all(np.abs(qd - qr) <= (0 if self.dtype == "f32" else 2.0 ** -8) * np.abs(qr) + 2.0 ** -20 * 8)
            ks, vs = self.stored(kr, self.sc.get("k_scale")), self.stored(h[2], self.sc.get("v_scale"))
            if self.dtype == "fp8":   # a rotated row next to a border may take the neighbouring code: use the cache's own
                ks = self.cached(kp, slots)
                assert np.all(np.abs(ks - kr) <= 2.0 ** -4 * np.abs(kr) * 1.01 + 2.0 ** -9 * self.sc["k_scale"])
            for i, r in enumerate(reqs):
                mine = rows == i
                self.k[r][layer] = np.concatenate([self.k[r][layer], ks[mine]])
                self.v[r][layer] = np.concatenate([self.v[r][layer], vs[mine]])
                want = self.attend(qd[mine], self.k[r][layer], self.v[r][layer])
                assert_close(to_f64(out)[mine], want, "f32" if self.dtype == "f32" else "bf16", f"layer {layer} request {r}")
        for r, n in zip(reqs, after):   # pages behind the window go back, the sinks' stay
            self.alloc.expire_window(r, max(0, n + 1 - WINDOW), SINKS)

    def cached(self, pool, slots):
        t, d = np.arange(BS)[:, None], np.arange(D)[None]
        kk = d % 16
        kb = (d // 64) * 1024 + (t // 8) * 512 + ((t % 8) * 4 + (kk % 8) // 2) * 16 + ((d % 64) // 16) * 4 + kk % 2 + 2 * (kk // 8)
        codes = pool.cpu().numpy()[(slots // BS)[:, None, None], np.arange(HKV)[None, :, None], kb[slots % BS][:, None, :]]
        return self.orc.e4m3_decode(codes.reshape(-1)).reshape(codes.shape) * self.sc["k_scale"]

    def attend(self, q, k, v):
        n, L = len(q), len(k)
        at, j = np.arange(L - n, L)[:, None], np.arange(L)[None]
        see = (j <= at) & ((j > at - WINDOW) | (j < SINKS))
        out = np.zeros((n, HQ, D))
        for h in range(HQ):
            s = np.where(see, q[:, h] @ k[:, h // (HQ // HKV)].T * D ** -0.5, -np.inf)
            p = np.exp(s - s.max(1, keepdims=True))
            out[:, h] = p @ v[:, h // (HQ // HKV)] / p.sum(1, keepdims=True)
        return out


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
def test_streams_forked_rolled_back_and_compacted(pkv, orc, dtype):
    s = Loop(pkv, orc, dtype, seed=1)
    a, b = s.begin(), s.begin()
    s.step({a: 70, b: 33})                       # chunked prefill, then decode
    s.step({a: 40, b: 90})
    for _ in range(3):
        s.step({a: 1, b: 1})
    n = len(s.k[a][0])
    c, pair = s.alloc.fork(a, n)                 # a beam: shares the full pages, owns the partial one
    s.copy([pair])
    s.k[c], s.v[c] = ([x.copy() for x in h[a]] for h in (s.k, s.v))
    for _ in range(20):                          # both go on, past a page's end
        s.step({a: 1, c: 1, b: 1})
    n = len(s.k[b][0])
    s.step({b: 4})                               # four speculated tokens, two of them rejected
    s.copy([s.alloc.truncate(b, n + 2)])
    for h in (s.k, s.v):
        h[b] = [x[:n + 2] for x in h[b]]
    s.step({a: 1, b: 1, c: 1})
    s.alloc.release(a)
    used = sum(s.alloc.refcount(i) > 0 for i in range(64))
    src, dst = s.alloc.compact(used)             # the pool shrinks to what is held
    s.copy(list(zip(src, dst)))
    assert s.alloc.stats()[0] == used
    s.step({b: 1, c: 1})                         # (the pool grows again as they go on)
    s.step({b: 30, c: 17})
    for _ in range(2):
        s.step({b: 1, c: 1})
