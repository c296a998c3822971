"""Rotary append (GPU) against the formula in extended precision.

Tolerance.  The sine and cosine are off by at most 2.2e-7 (the fixed-point
angle rounded to fp32 in half turns: pi 2^-25; two ulps of sincospif), the
factor and the two products add four roundings of 2^-24: together under
2^-21 (|x1| + |x2|) |factor|.  bf16 results add their own rounding, 2^-8 |y|;
E4M3 codes half a step: 2^-4 |y|, or half the subnormal spacing 2^-10 scale.
"""
import numpy as np
import pytest

import pkv_inputs as gen
from gpu_util import storage_bytes, to_f64, to_torch

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KS, VS = float(gen.FP8_K_SCALE), float(gen.FP8_V_SCALE)


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_paged_kv_gb300 as m
    return m


def inv_freq(rd, base=10000.0):
    return base ** (-2.0 * np.arange(rd // 2) / rd)


def rotate(x, pos, freq, axis, interleaved, factor):
    """x [T, H, D] float64: the rotated rows, and |x1| + |x2| of each element's pair."""
    n = len(freq)
    th = pos[axis].T.astype(np.longdouble) * freq.astype(np.longdouble)      # [T, n]
    th = np.remainder(th, 2 * np.longdouble("3.14159265358979323846264338327950288"))
    c, s = np.cos(th).astype(np.float64)[:, None], np.sin(th).astype(np.float64)[:, None]
    y, mag = x.copy(), np.zeros_like(x)
    a, b = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    y[..., a] = factor * (x[..., a] * c - x[..., b] * s)
    y[..., b] = factor * (x[..., b] * c + x[..., a] * s)
    mag[..., a] = mag[..., b] = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(factor)
    return y, mag


def k_tile_bytes(D):
    """Byte of (token, dim) in an FP8 K tile."""
    t, d = np.arange(16)[:, None], np.arange(D)[None]
    k = d % 16
    return (d // 64) * 1024 + (t // 8) * 512 + ((t % 8) * 4 + (k % 8) // 2) * 16 + ((d % 64) // 16) * 4 \
        + k % 2 + 2 * (k // 8)


class Case:
    def __init__(self, seed, dtype, T, hq, hkv, D, axes=1, rd=None, far=3000, bs=16, order="runs"):
        self.dtype, self.T, self.hq, self.hkv, self.D, self.bs = dtype, T, hq, hkv, D, bs
        rng = np.random.default_rng(seed)
        self.nb = -(-T // bs) + 5
        self.bits = bits = "f32" if dtype == "f32" else "bf16"
        self.q = gen._values(seed, "q", (T, hq, D), bits)
        self.k = gen._values(seed, "k", (T, hkv, D), bits)
        self.v = gen._values(seed, "v", (T, hkv, D), bits)
        if order == "runs":      # runs of tokens through shuffled pages, from inside a page
            at = int(rng.integers(0, bs)) + np.arange(T)
            self.slots = (rng.permutation(self.nb)[at // bs] * bs + at % bs).astype(np.int32)
        else:                    # tokens anywhere
            self.slots = rng.permutation(self.nb * bs)[:T].astype(np.int32)
        self.pos = rng.integers(0, far, size=(axes, T)).astype(np.int32)
        self.rd = rd or D
        self.axis = np.arange(self.rd // 2) * axes // (self.rd // 2)
        if dtype == "fp8":
            self.kp, self.vp = (np.full((self.nb, hkv, 16 * D), gen.FP8_POISON, np.uint8) for _ in range(2))
        else:
            shape = (self.nb, hkv, bs, D)
            self.kp, self.vp = gen._values(seed, "kp", shape, bits), gen._values(seed, "vp", shape, bits)
        self.scales = dict(k_scale=KS, v_scale=VS) if dtype == "fp8" else {}

    def dev(self):
        up = (lambda a: torch.from_numpy(a.copy()).cuda()) if self.dtype == "fp8" else (lambda a: to_torch(a, self.bits))
        return up(self.kp), up(self.vp)


def run(pkv, c, interleaved=False, factor=1.0, freq=None):
    freq = inv_freq(c.rd) if freq is None else freq
    rope = pkv.make_rope(freq, c.axis, num_axes=c.pos.shape[0], interleaved=interleaved, factor=factor)
    kp, vp = c.dev()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = pkv.paged_kv_append_rope(kp, vp, torch.from_numpy(c.slots).cuda(), to_torch(c.q, c.bits),
                                     to_torch(c.k, c.bits), to_torch(c.v, c.bits),
                                     torch.from_numpy(c.pos).cuda(), rope, status=status, **c.scales)
    torch.cuda.synchronize()
    return q_out, kp, vp, int(status.item())


def check(pkv, orc, c, interleaved=False, factor=1.0, freq=None):
    freq = inv_freq(c.rd) if freq is None else freq
    q_out, kp, vp, status = run(pkv, c, interleaved, factor, freq)
    assert status == 0
    own = 0.0 if c.dtype == "f32" else 2.0 ** -8
    x = gen.as_f32(c.q, c.bits).astype(np.float64)
    y, mag = rotate(x, c.pos, freq, c.axis, interleaved, factor)
    err = np.abs(to_f64(q_out) - y)
    assert np.all(err <= own * np.abs(y) + 2.0 ** -21 * mag), err.max()
    assert np.array_equal(to_f64(q_out)[..., c.rd:], x[..., c.rd:])      # dims past the rotary ones: copied
    xk = gen.as_f32(c.k, c.bits).astype(np.float64)
    yk, magk = rotate(xk, c.pos, freq, c.axis, interleaved, factor)
    live = c.slots >= 0
    s = c.slots[live]
    ref_k, ref_v = c.kp.copy(), c.vp.copy()
    orc.append(ref_k, ref_v, "fp8" if c.dtype == "fp8" else c.bits, c.slots, c.k, c.v, **c.scales)
    assert storage_bytes(vp) == ref_v.tobytes()                            # V: the plain append's bytes
    if c.dtype == "fp8":
        at = ((s // 16)[:, None, None], np.arange(c.hkv)[None, :, None], k_tile_bytes(c.D)[s % 16][:, None, :])
        got = kp.cpu().numpy()
        codes = got[at]
        val = orc.e4m3_decode(codes.reshape(-1)).reshape(codes.shape) * KS
        want = np.clip(yk[live], -448 * KS, 448 * KS)
        err = np.abs(val - want)
        assert np.all(err <= 2.0 ** -4 * np.abs(want) + 2.0 ** -10 * KS + 2.0 ** -21 * magk[live]), err.max()
        rest = np.ones(c.kp.shape, bool)
        rest[at] = False
        assert np.array_equal(got[rest], c.kp[rest])                        # other slots untouched
    else:
        val = to_f64(kp)
        err = np.abs(val[s // c.bs, :, s % c.bs] - yk[live])
        assert np.all(err <= own * np.abs(yk[live]) + 2.0 ** -21 * magk[live]), err.max()
        rest = np.ones((c.nb, c.bs), bool)
        rest[s // c.bs, s % c.bs] = False
        at = np.broadcast_to(rest[:, None, :, None], val.shape)
        assert np.array_equal(val[at], gen.as_f32(c.kp, c.bits).astype(np.float64)[at])


@pytest.mark.parametrize("dtype,D", [("f32", 32), ("f32", 64), ("bf16", 64), ("bf16", 80), ("bf16", 128),
                                     ("bf16", 256), ("fp8", 64), ("fp8", 128), ("fp8", 256)])
@pytest.mark.parametrize("T", [1, 7, 33, 300])
@pytest.mark.parametrize("interleaved", [False, True])
def test_types_dims_lengths(pkv, orc, dtype, D, T, interleaved):
    check(pkv, orc, Case(400 + D + T, dtype, T, 4, 2, D, axes=1 + 2 * (T % 2)), interleaved)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("rd", [16, 32, 48, 96, 112])
@pytest.mark.parametrize("interleaved", [False, True])
def test_partial_rotary(pkv, orc, dtype, rd, interleaved):
    check(pkv, orc, Case(410 + rd, dtype, 40, 3, 3, 128, axes=2, rd=rd), interleaved)
    check(pkv, orc, Case(411 + rd, dtype, 1300, 1, 1, 128, axes=1, rd=rd), interleaved)


@pytest.mark.parametrize("dtype", ["bf16", "fp8"])
@pytest.mark.parametrize("hq,hkv", [(32, 8), (1, 1), (9, 9), (40, 5)])
@pytest.mark.parametrize("T,order", [(2500, "runs"), (1500, "anywhere"), (20, "anywhere"), (160, "runs")])
def test_heads_and_long_runs(pkv, orc, dtype, hq, hkv, T, order):
    check(pkv, orc, Case(420 + hq + T, dtype, T, hq, hkv, 128, axes=3, order=order))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_far_and_negative_positions(pkv, orc, dtype):
    # to the ends of int32 (a table entry's rounding, 2^-65 turns, adds 4e-10 rad there)
    c = Case(430, dtype, 64, 4, 2, 128, axes=2)
    c.pos[:] = np.random.default_rng(430).integers(-2 ** 31, 2 ** 31, size=c.pos.shape)
    c.pos[0, :4] = [2 ** 31 - 1, -2 ** 31, 0, -1]
    check(pkv, orc, c)
    check(pkv, orc, c, freq=np.concatenate([[3.0, -2.5, 1e-9, 0.0, 100.25], inv_freq(128, 1e7)[5:]]))


@pytest.mark.parametrize("dtype,bs", [("f32", 16), ("bf16", 16), ("fp8", 16), ("bf16", 8), ("f32", 24)])
@pytest.mark.parametrize("T", [77, 1400])
def test_position_zero_is_the_plain_append(pkv, orc, dtype, bs, T):
    c = Case(440, dtype, T, 4, 2, 64, bs=bs)
    c.pos[:] = 0
    q_out, kp, vp, status = run(pkv, c)
    ref_k, ref_v = c.kp.copy(), c.vp.copy()
    orc.append(ref_k, ref_v, "fp8" if dtype == "fp8" else c.bits, c.slots, c.k, c.v, **c.scales)
    assert status == 0 and storage_bytes(q_out) == c.q.tobytes()
    assert storage_bytes(kp) == ref_k.tobytes() and storage_bytes(vp) == ref_v.tobytes()


def test_fp8_paths_store_the_same_codes(pkv):
    # the tokens of one long call, again in short calls: whatever path a call
    # takes, an element is rotated and quantized by the same operations
    c = Case(441, "fp8", 1400, 4, 2, 128, axes=3)
    q_out, kp, vp, _ = run(pkv, c)
    rope = pkv.make_rope(inv_freq(128), c.axis, num_axes=3)
    k2, v2 = c.dev()
    q2 = torch.empty_like(q_out)
    for a in range(0, 1400, 100):
        sl = slice(a, a + 100)
        pkv.paged_kv_append_rope(k2, v2, torch.from_numpy(c.slots[sl]).cuda(), to_torch(c.q[sl], "bf16"),
                                 to_torch(c.k[sl], "bf16"), to_torch(c.v[sl], "bf16"),
                                 torch.from_numpy(np.ascontiguousarray(c.pos[:, sl])).cuda(), rope,
                                 q_out=q2[sl], **c.scales)
    assert torch.equal(q2, q_out) and torch.equal(k2, kp) and torch.equal(v2, vp)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
def test_factor(pkv, orc, dtype):
    check(pkv, orc, Case(450, dtype, 30, 4, 2, 64), factor=1.375)
    check(pkv, orc, Case(451, dtype, 30, 4, 2, 64, rd=32), interleaved=True, factor=-0.5)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("T", [40, 1500])
def test_skipped_and_bad_slots(pkv, orc, dtype, T):
    c = Case(460, dtype, T, 4, 2, 64)
    c.slots[::37] = -1
    check(pkv, orc, c)           # q is rotated all the same; skipped slots untouched
    c.slots[1] = c.nb * c.bs
    q_out, kp, vp, status = run(pkv, c)
    assert status == pkv.DEV_BAD_SLOT
    c.slots[1] = -1
    q2, k2, v2, _ = run(pkv, c)
    assert torch.equal(q_out, q2) and torch.equal(kp, k2) and torch.equal(vp, v2)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "fp8"])
@pytest.mark.parametrize("T", [1, 50, 1400])
def test_rows_cut_from_a_projection_and_in_place(pkv, dtype, T):
    c = Case(470, dtype, T, 6, 2, 128, axes=3)
    want_q, want_k, want_v, _ = run(pkv, c)
    act = torch.float32 if dtype == "f32" else torch.bfloat16
    wide = torch.zeros(T, (6 + 2 + 2) * 128 + 64, dtype=act, device="cuda")
    q, k, v = wide[:, :768].view(T, 6, 128), wide[:, 768:1024].view(T, 2, 128), wide[:, 1024:1280].view(T, 2, 128)
    for view, rows in ((q, c.q), (k, c.k), (v, c.v)):
        view.copy_(to_torch(rows, c.bits))
    rope = pkv.make_rope(inv_freq(128), c.axis, num_axes=3)
    kp, vp = c.dev()
    pos = torch.zeros(3, T + 9, dtype=torch.int32, device="cuda")
    pos[:, :T] = torch.from_numpy(c.pos).cuda()
    out = pkv.paged_kv_append_rope(kp, vp, torch.from_numpy(c.slots).cuda(), q, k, v, pos[:, :T], rope, q_out=q,
                                   **c.scales)
    assert out is q
    assert torch.equal(q, want_q) and torch.equal(kp, want_k) and torch.equal(vp, want_v)
    assert torch.equal(wide[:, 1280:], torch.zeros_like(wide[:, 1280:]))


def test_k_alone_and_no_tokens(pkv):
    c = Case(480, "bf16", 50, 4, 2, 128)
    _, want_k, want_v, _ = run(pkv, c)
    rope = pkv.make_rope(inv_freq(128))
    kp, vp = c.dev()
    a = (torch.from_numpy(c.slots).cuda(), None, to_torch(c.k, "bf16"), to_torch(c.v, "bf16"),
         torch.from_numpy(c.pos[0]).cuda())
    assert pkv.paged_kv_append_rope(kp, vp, *a, rope) is None
    assert torch.equal(kp, want_k) and torch.equal(vp, want_v)
    n0 = pkv.launch_count()
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    none = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    assert pkv.paged_kv_append_rope(kp, vp, e, none, none, none, e, rope).shape == (0, 2, 128)
    assert pkv.launch_count() == n0


def test_nan_and_inf_stay_in_their_pair(pkv):
    c = Case(481, "bf16", 40, 4, 2, 64)
    c.q[3, 1, 5], c.k[7, 0, 9] = gen.BF16_NAN, 0x7F80
    q_out, kp, vp, _ = run(pkv, c)
    bad = torch.zeros(40, 4, 64, dtype=torch.bool)
    bad[3, 1, 5] = bad[3, 1, 37] = True
    assert torch.equal(torch.isnan(q_out).cpu(), bad)
    s = int(c.slots[7])
    hit = ~torch.isfinite(kp[s // 16, 0, s % 16].float().cpu())
    assert hit[9] and hit[41] and int(hit.sum()) == 2


def test_captured_and_replayed_on_another_stream(pkv):
    c = Case(482, "bf16", 32, 8, 2, 128, axes=3)
    want_q, want_k, _, _ = run(pkv, c)
    rope = pkv.make_rope(inv_freq(128), c.axis, num_axes=3)
    kp, vp = c.dev()
    a = [torch.from_numpy(c.slots).cuda(), to_torch(c.q, "bf16"), to_torch(c.k, "bf16"), to_torch(c.v, "bf16"),
         torch.from_numpy(c.pos).cuda()]
    q_out = torch.empty_like(a[1])
    pos = a[4].clone()
    a[4].zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_kv_append_rope(kp, vp, *a, rope, q_out=q_out)
    rope._c.freq[0] = 0          # the descriptor went into the launch by value
    a[4].copy_(pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(q_out, want_q) and torch.equal(kp, want_k)


def test_refusals(pkv):
    c = Case(490, "bf16", 20, 4, 2, 128, axes=2)
    kp, vp = c.dev()
    slots, pos = torch.from_numpy(c.slots).cuda(), torch.from_numpy(c.pos).cuda()
    q, k, v = (to_torch(x, "bf16") for x in (c.q, c.k, c.v))
    rope = pkv.make_rope(inv_freq(128), c.axis)
    n0 = pkv.launch_count()
    for bad in (dict(q=q.float()), dict(k=k[:10]), dict(pos=pos[:1]), dict(pos=pos.long()),
                dict(pos=pos.t().contiguous().t()), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(v=v.cpu()), dict(slots=slots.long()), dict(q_out=torch.empty_like(q).cpu()),
                dict(q_out=q[:, :2]), dict(q=None, q_out=q)):
        a = dict(slots=slots, q=q, k=k, v=v, pos=pos, q_out=None) | bad
        with pytest.raises(ValueError):
            pkv.paged_kv_append_rope(kp, vp, a["slots"], a["q"], a["k"], a["v"], a["pos"], rope, q_out=a["q_out"])
    flat = torch.zeros(20 * 4 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(pkv.PkvError) as e:      # 2 bytes off a 16-byte boundary
        pkv.paged_kv_append_rope(kp, vp, slots, flat[1:-7].view(20, 4, 128), k, v, pos, rope)
    assert e.value.code == pkv.PKV_ERR_INVALID_ARG
    for rd, code in ((24, pkv.PKV_ERR_UNSUPPORTED), (256, pkv.PKV_ERR_INVALID_ARG)):
        with pytest.raises(pkv.PkvError) as e:  # not whole vectors; wider than the head
            pkv.paged_kv_append_rope(kp, vp, slots, q, k, v, pos, pkv.make_rope(inv_freq(rd), num_axes=2))
        assert e.value.code == code
    assert pkv.launch_count() == n0
