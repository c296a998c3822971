"""Sliding window with sink tokens (GPU): decode, verify steps, chunked prefill
and grouped decode against dense attention in 64 bits over the visible keys.

Every pool slot that no query of a row may see (between the sinks and the
window, past the length, unreferenced blocks) holds NaN, and table entries of
blocks without a visible position hold -1.  Tolerances are the framework's:
bf16 |gpu - ref| <= 2e-3 + 1e-2 |ref| (the output's own rounding is 2^-8 |ref|),
f32 1e-5 + 1e-5 |ref|.
"""
import dataclasses

import numpy as np
import pytest

import pkv_inputs as gen
from gpu_util import Dev, append, assert_close, to_f64

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_paged_kv_gb300 as m
    return m


def queries(w, r):
    return (int(w.cu_q_lens[r]), int(w.cu_q_lens[r + 1])) if w.cu_q_lens is not None else (r, r + 1)


def visible(w, r, sinks):
    """Positions of row r that any of its queries sees."""
    q0, q1 = queries(w, r)
    L = int(w.seq_lens[r])
    j = np.arange(L if q1 > q0 else 0)
    return j[(j < sinks) | (j > L - (q1 - q0) - w.window)]


def reference(w, sinks, k_rows, v_rows):
    """Dense attention in 64 bits; k_rows(r, positions) -> [n, Hkv, D] float64."""
    q = torch.from_numpy(gen.as_f32(w.q, w.dtype)).double()
    out = torch.zeros(q.shape, dtype=torch.float64)
    G = w.num_q_heads // w.num_kv_heads
    for r in range(w.batch):
        L = int(w.seq_lens[r])
        q0, q1 = queries(w, r)
        pos = visible(w, r, sinks)
        if L == 0 or q1 == q0:
            continue
        K, V = torch.from_numpy(k_rows(r, pos)), torch.from_numpy(v_rows(r, pos))
        at = torch.arange(L - (q1 - q0), L)[:, None]
        j = torch.from_numpy(pos)[None]
        see = (j <= at) & ((j > at - w.window) | (j < sinks))
        s = torch.einsum("chgd,nhd->hgcn", q[q0:q1].view(q1 - q0, w.num_kv_heads, G, -1), K) * w.scale
        p = torch.softmax(s.masked_fill(~see, -float("inf")), -1)
        out[q0:q1] = torch.einsum("hgcn,nhd->chgd", p, V).reshape(q1 - q0, w.num_q_heads, -1)
    return out.numpy()


def pool_rows(w, pool):
    def rows(r, pos):
        b = w.block_tables[r, pos // w.block_size]
        return gen.as_f32(pool[b, :, pos % w.block_size], w.dtype).astype(np.float64)
    return rows


def hide(w, sinks):
    """NaN in every slot without a visible position, -1 for blocks without one."""
    seen = np.zeros((w.num_blocks, w.block_size), dtype=bool)
    held = np.zeros(w.block_tables.shape, dtype=bool)
    for r in range(w.batch):
        pos = visible(w, r, sinks)
        seen[w.block_tables[r, pos // w.block_size], pos % w.block_size] = True
        held[r, pos // w.block_size] = True
    nan = gen.BF16_NAN if w.dtype == "bf16" else gen.F32_NAN
    for pool in (w.k_pool, w.v_pool):
        pool[np.broadcast_to(~seen[:, None, :], pool.shape[:3])] = nan
    w.block_tables[~held] = -1


def setup(pkv, orc, w, sinks):
    """Append the new rows, then hide what no query may see."""
    slots = pkv.slot_mapping_host(w.block_tables, w.num_blocks, w.new_rows, w.new_pos, w.block_size)
    orc.append(w.k_pool, w.v_pool, w.dtype, slots, w.k_new, w.v_new)
    hide(w, sinks)
    return Dev(w)


def call(pkv, w, d, sinks, kp=None, vp=None, **kw):
    kp, vp = (d.k_pool, d.v_pool) if kp is None else (kp, vp)
    kw = dict(max_seq_len=int(w.seq_lens.max()), status=d.status, sinks=sinks) | kw
    if w.cu_q_lens is None:
        return pkv.paged_decode_attention(d.q, kp, vp, d.tables, d.seq_lens, w.window, w.scale, **kw)
    return pkv.paged_prefill_chunk_attention(d.q, d.cu, kp, vp, d.tables, d.seq_lens,
                                             int(np.max(np.diff(w.cu_q_lens))), w.window, w.scale, **kw)


def check(pkv, orc, w, sinks):
    d = setup(pkv, orc, w, sinks)
    out = call(pkv, w, d, sinks)
    torch.cuda.synchronize()
    assert int(d.status.item()) == 0
    ref = reference(w, sinks, pool_rows(w, w.k_pool), pool_rows(w, w.v_pool))
    assert_close(to_f64(out), ref, w.dtype, f"{w.dtype} sinks {sinks} window {w.window}")
    assert torch.equal(out, call(pkv, w, d, sinks))   # the cut depends on sizes alone


CTX = [0, 1, 14, 15, 16, 60, 100, 333, 700]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 4), (128, 8, 2), (256, 8, 1), (64, 16, 1), (128, 6, 2), (256, 16, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (37, 4), (64, 16), (200, 21), (50, 640), (16, 33)])
def test_decode_shapes(pkv, orc, dtype, d, hq, hkv, window, sinks):
    check(pkv, orc, gen.decode_workload(seed=300 + d + hq + window, dtype=dtype, num_q_heads=hq,
                                        num_kv_heads=hkv, head_dim=d, context_lens=CTX, window=window), sinks)


@pytest.mark.parametrize("window,sinks", [(5, 100000), (1 << 30, 7), (5, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 1)])
def test_more_sinks_or_window_than_tokens(pkv, orc, window, sinks):
    check(pkv, orc, gen.decode_workload(seed=310, dtype="bf16", num_q_heads=8, num_kv_heads=2, head_dim=128,
                                        context_lens=[0, 40, 333], window=window), sinks)
    check(pkv, orc, gen.prefill_workload(seed=310, dtype="bf16", num_q_heads=8, num_kv_heads=2, head_dim=128,
                                         prefix_lens=[0, 100], chunk_lens=[40, 90], window=window), sinks)


@pytest.mark.parametrize("dtype,d,hq,hkv,batch,window", [
    ("bf16", 128, 32, 8, 1, 4000), ("bf16", 128, 8, 8, 40, 500), ("bf16", 256, 8, 1, 4, 512),
    ("bf16", 64, 6, 2, 70, 300), ("f32", 64, 4, 2, 40, 700), ("bf16", 128, 4, 1, 2, 9000)])
def test_decode_many_splits_and_rows(pkv, orc, dtype, d, hq, hkv, batch, window):
    ctx = [int(x) for x in gen.uniform_ints(311, "ctx", batch, 0, 2 * window)]
    check(pkv, orc, gen.decode_workload(seed=311 + d, dtype=dtype, num_q_heads=hq, num_kv_heads=hkv,
                                        head_dim=d, context_lens=ctx, window=window), 20)


@pytest.mark.parametrize("scale", [-0.3, 0.0])
def test_scale_sign_and_zero(pkv, orc, scale):
    w = gen.decode_workload(seed=312, dtype="bf16", num_q_heads=8, num_kv_heads=2, head_dim=128,
                            context_lens=[1, 30, 300], window=40)
    check(pkv, orc, dataclasses.replace(w, scale=scale), 5)


def test_far_stream_reads_only_live_blocks(pkv):
    # a row a million tokens long that holds its sinks and its window alone
    L, window, sinks, bs = 1_000_003, 100, 6, 16
    w = gen.decode_workload(seed=313, dtype="bf16", num_q_heads=8, num_kv_heads=2, head_dim=128,
                            context_lens=[200], window=window)
    d = Dev(w)
    append(pkv, d)
    d.k_pool.nan_to_num_()
    d.v_pool.nan_to_num_()
    tables = torch.full((1, -(-L // bs)), -1, dtype=torch.int32, device="cuda")
    first = (L - window) // bs
    ids = [int(x) for x in w.block_tables[0, :1 + tables.shape[1] - first]]
    tables[0, 0] = ids[0]
    tables[0, first:] = torch.tensor(ids[1:], dtype=torch.int32, device="cuda")
    out = pkv.paged_decode_attention(d.q, d.k_pool, d.v_pool, tables,
                                     torch.tensor([L], dtype=torch.int32, device="cuda"), window, w.scale,
                                     status=d.status, sinks=sinks)
    torch.cuda.synchronize()
    assert int(d.status.item()) == 0
    pos = np.concatenate([np.arange(sinks), np.arange(L - window, L)])
    tab = tables.cpu().numpy()[0]
    K, V = (x.float().cpu().numpy()[tab[pos // bs], :, pos % bs].astype(np.float64) for x in (d.k_pool, d.v_pool))
    q = gen.as_f32(w.q, "bf16").astype(np.float64)[0]
    for h in range(8):
        s = K[:, h // 4] @ q[h] * w.scale
        p = np.exp(s - s.max())
        assert_close(to_f64(out)[0, h], p @ V[:, h // 4] / p.sum(), "bf16", "far stream")


@pytest.mark.parametrize("hq,hkv", [(8, 4), (32, 8), (16, 1)])
@pytest.mark.parametrize("window,sinks", [(50, 4), (130, 70), (64, 1000), (1, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_ragged(pkv, orc, dtype, hq, hkv, window, sinks):
    check(pkv, orc, gen.prefill_workload(seed=320 + hq + window, dtype=dtype, num_q_heads=hq,
                                         num_kv_heads=hkv, head_dim=128, prefix_lens=[0, 5, 130, 300, 1],
                                         chunk_lens=[1, 47, 200, 129, 0], window=window), sinks)


@pytest.mark.parametrize("chunks", [[3, 1, 4, 2], [20, 33, 5, 32], [600, 300, 1, 520]])
def test_prefill_schedules(pkv, orc, chunks):
    # verify steps on the decode kernel, one query tile cut into key runs, and
    # chunks of several query tiles; windows long enough for many key tiles
    check(pkv, orc, gen.prefill_workload(seed=330 + chunks[0], dtype="bf16", num_q_heads=16, num_kv_heads=4,
                                         head_dim=128, prefix_lens=[3000, 40, 2500, 1200], chunk_lens=chunks,
                                         window=1000), 70)


@pytest.mark.parametrize("window,sinks", [(150, 9), (700, 200)])
def test_prefill_balanced_schedule(pkv, orc, window, sinks):
    # more (row, kv head, query-tile pair) items than SMs
    check(pkv, orc, gen.prefill_workload(seed=334, dtype="bf16", num_q_heads=16, num_kv_heads=4, head_dim=128,
                                         prefix_lens=[0, 300, 1700, 90] * 10, chunk_lens=[70, 33, 64, 128] * 10,
                                         window=window), sinks)


@pytest.mark.parametrize("d,q_len", [(64, 2), (128, 4), (256, 3)])
@pytest.mark.parametrize("window,sinks", [(1, 3), (40, 17), (300, 5)])
def test_verify_steps(pkv, orc, d, q_len, window, sinks):
    check(pkv, orc, gen.prefill_workload(seed=340 + d, dtype="bf16", num_q_heads=8, num_kv_heads=2, head_dim=d,
                                         prefix_lens=[0, 3, 90, 500], chunk_lens=[q_len, 1, q_len, q_len],
                                         window=window), sinks)


def check_fp8(pkv, orc, w, sinks):
    """The workload's context and new rows in FP8 pools; hidden slots hold the NaN code."""
    sc = dict(k_scale=float(gen.FP8_K_SCALE), v_scale=float(gen.FP8_V_SCALE))
    kp, vp = gen.fp8_empty_pools(w)
    slots, kr, vr = gen.live_slots(w)
    new = pkv.slot_mapping_host(w.block_tables, w.num_blocks, w.new_rows, w.new_pos, 16)
    slots, kr, vr = np.concatenate([slots, new]), np.concatenate([kr, w.k_new]), np.concatenate([vr, w.v_new])
    seen = np.zeros(w.num_blocks * 16, dtype=bool)
    for r in range(w.batch):
        pos = visible(w, r, sinks)
        seen[w.block_tables[r, pos // 16] * 16 + pos % 16] = True
    orc.append(kp, vp, "fp8", slots[seen[slots]], kr[seen[slots]], vr[seen[slots]], **sc)
    rows, tables = [], w.block_tables.copy()
    for x, s in ((kr, sc["k_scale"]), (vr, sc["v_scale"])):
        q = (gen.bf16_to_f32(x) / np.float32(s)).astype(np.float32)
        flat = np.full((w.num_blocks * 16, w.num_kv_heads, w.head_dim), np.nan)
        flat[slots] = orc.e4m3_decode(orc.e4m3_encode(q.reshape(-1))).reshape(q.shape) * s
        rows.append(lambda r, p, flat=flat: flat[tables[r, p // 16] * 16 + p % 16])
    hide(w, sinks)
    d = Dev(w)
    kd, vd = torch.from_numpy(kp).cuda(), torch.from_numpy(vp).cuda()
    out = call(pkv, w, d, sinks, kd, vd, **sc)
    torch.cuda.synchronize()
    assert int(d.status.item()) == 0
    assert_close(to_f64(out), reference(w, sinks, *rows), "bf16", f"fp8 sinks {sinks} window {w.window}")
    assert torch.equal(out, call(pkv, w, d, sinks, kd, vd, **sc))


@pytest.mark.parametrize("d,hq,hkv", [(64, 4, 4), (128, 8, 2), (256, 8, 1), (128, 16, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 1), (37, 4), (200, 21), (50, 640)])
def test_fp8_decode(pkv, orc, d, hq, hkv, window, sinks):
    check_fp8(pkv, orc, gen.decode_workload(seed=350 + d + hq, dtype="bf16", num_q_heads=hq, num_kv_heads=hkv,
                                            head_dim=d, context_lens=CTX + [2000], window=window), sinks)


@pytest.mark.parametrize("hq,hkv", [(8, 4), (32, 8), (16, 1)])
@pytest.mark.parametrize("window,sinks", [(50, 4), (130, 70), (1000, 9)])
@pytest.mark.parametrize("chunks", [[1, 47, 200, 129], [3, 1, 2, 1]])
def test_fp8_prefill(pkv, orc, hq, hkv, window, sinks, chunks):
    check_fp8(pkv, orc, gen.prefill_workload(seed=360 + hq, dtype="bf16", num_q_heads=hq, num_kv_heads=hkv,
                                             head_dim=128, prefix_lens=[0, 5, 130, 1500], chunk_lens=chunks,
                                             window=window), sinks)


def test_no_sinks_and_no_window_are_the_plain_calls(pkv):
    w = gen.decode_workload(seed=370, dtype="bf16", num_q_heads=8, num_kv_heads=2, head_dim=128,
                            context_lens=[100, 700], window=0)
    d = Dev(w)
    append(pkv, d)
    a = (d.q, d.k_pool, d.v_pool, d.tables, d.seq_lens)
    assert torch.equal(pkv.paged_decode_attention(*a, 0, w.scale, sinks=5),
                       pkv.paged_decode_attention(*a, 0, w.scale))
    assert torch.equal(pkv.paged_decode_attention(*a, 64, w.scale, sinks=0),
                       pkv.paged_decode_attention(*a, 64, w.scale))


@pytest.mark.parametrize("batch", [3, 40])
def test_groups_with_sinks_equal_their_own_calls(pkv, batch):
    groups, own = [], []
    for i, (window, sinks) in enumerate(((0, 0), (64, 4), (100, 0), (30, 40))):
        w = gen.decode_workload(seed=380 + i, dtype="bf16", num_q_heads=8, num_kv_heads=1, head_dim=256,
                                context_lens=([100, 700, 31] * batch)[:batch], window=window)
        d = Dev(w)
        append(pkv, d)
        groups.append(pkv.DecodeGroup(d.q, d.k_pool, d.v_pool, d.tables, d.seq_lens, window, w.scale, sinks=sinks))
        own.append(pkv.paged_decode_attention(d.q, d.k_pool, d.v_pool, d.tables, d.seq_lens, window,
                                              w.scale, sinks=sinks))
    for got, want in zip(pkv.paged_decode_attention_groups(groups), own):
        assert torch.equal(got, want)
    # every group with sinks: nothing is left for the fused launch
    for got, want in zip(pkv.paged_decode_attention_groups([groups[1], groups[3]]), [own[1], own[3]]):
        assert torch.equal(got, want)


def test_captured_and_replayed(pkv):
    w = gen.decode_workload(seed=390, dtype="bf16", num_q_heads=8, num_kv_heads=2, head_dim=128,
                            context_lens=[100, 700], window=64)
    d = Dev(w)
    append(pkv, d)
    out = torch.empty_like(d.q)
    ws = pkv.alloc_workspace(pkv.decode_workspace_size(2, 8, 2, 128, 16, 704, 64, sinks=4), "cuda")

    def step():
        pkv.paged_decode_attention(d.q, d.k_pool, d.v_pool, d.tables, d.seq_lens, 64, w.scale, out=out,
                                   workspace=ws, max_seq_len=704, sinks=4)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    d.seq_lens.copy_(torch.tensor([90, 650], dtype=torch.int32))   # replays follow the device's lengths
    g.replay()
    torch.cuda.synchronize()
    got = out.clone()
    step()
    torch.cuda.synchronize()
    assert torch.equal(got, out)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_missing_block_in_range_sets_status(pkv, dtype):
    w = gen.decode_workload(seed=391, dtype=dtype, num_q_heads=8, num_kv_heads=2, head_dim=128,
                            context_lens=[500], window=64)
    d = Dev(w)
    append(pkv, d)
    d.tables[0, 0] = -1                # the sinks' block
    out = call(pkv, w, d, 4)
    torch.cuda.synchronize()
    assert int(d.status.item()) == pkv.DEV_BAD_BLOCK and torch.isfinite(out.float()).all()
    d.tables[0, 0] = w.num_blocks + 3
    d.seq_lens[0] = 10000              # past the table: clamped
    call(pkv, w, d, 4)
    torch.cuda.synchronize()
    assert int(d.status.item()) & pkv.DEV_BAD_LEN


@pytest.mark.parametrize("d,batch", [(128, 3), (256, 60)])
@pytest.mark.parametrize("fp8", [False, True])
def test_wait_timeout_drill(pkv, d, batch, fp8):
    # every pipeline's first load is withheld: the waits run out, the call
    # returns with the status bit, and the next call is clean
    w = gen.decode_workload(seed=393, dtype="bf16", num_q_heads=8, num_kv_heads=1, head_dim=d,
                            context_lens=([300, 700, 64] * batch)[:batch], window=250)
    dev = Dev(w)
    kw, kp, vp = {}, dev.k_pool, dev.v_pool
    append(pkv, dev)
    if fp8:
        kp, vp = pkv.fp8_pools(w.num_blocks, 1, d, "cuda")
        kw = dict(k_scale=1.0, v_scale=1.0)
    want = call(pkv, w, dev, 20, kp, vp, **kw).clone()
    pkv.set_wait_drill(1_000_000, pkv.DRILL_WITHHOLD_FIRST_LOAD)
    try:
        call(pkv, w, dev, 20, kp, vp, **kw)
        torch.cuda.synchronize()
    finally:
        pkv.set_wait_drill()
    assert int(dev.status.item()) & pkv.DEV_TIMEOUT
    dev.status.zero_()
    out = call(pkv, w, dev, 20, kp, vp, **kw)
    torch.cuda.synchronize()
    assert int(dev.status.item()) == 0 and torch.equal(out, want)


def test_refusals(pkv):
    w = gen.decode_workload(seed=392, dtype="bf16", num_q_heads=8, num_kv_heads=2, head_dim=128,
                            context_lens=[500, 500], window=64)
    d = Dev(w)
    a = (d.q, d.k_pool, d.v_pool, d.tables, d.seq_lens)
    big = pkv.alloc_workspace(1 << 20, "cuda")
    n0 = pkv.launch_count()
    desc = pkv.PrefixDesc(1, 2, 1, torch.zeros(2, dtype=torch.int32, device="cuda"),
                          torch.ones(1, dtype=torch.int32, device="cuda"))
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    for code, fn in (
            (pkv.PKV_ERR_INVALID_ARG, lambda: pkv.paged_decode_attention(*a, 64, w.scale, sinks=-1, workspace=big)),
            (pkv.PKV_ERR_INVALID_ARG, lambda: pkv.paged_decode_attention(*a, 0, w.scale, sinks=-1, workspace=big)),
            (pkv.PKV_ERR_WORKSPACE, lambda: pkv.paged_decode_attention(*a, 64, w.scale, sinks=4, workspace=big[:256])),
            (pkv.PKV_ERR_WORKSPACE, lambda: pkv.paged_decode_attention(*a, 64, w.scale, sinks=4, workspace=big[16:])),
            (pkv.PKV_ERR_UNSUPPORTED, lambda: pkv.paged_decode_attention(*a, 64, w.scale, sinks=4, prefix=desc)),
            (pkv.PKV_ERR_INVALID_ARG, lambda: pkv.paged_prefill_chunk_attention(
                d.q, cu, *a[1:], 1, 64, w.scale, sinks=-3, workspace=big)),
            (pkv.PKV_ERR_INVALID_ARG, lambda: pkv.paged_decode_attention_groups(
                [pkv.DecodeGroup(*a, 64, w.scale, sinks=-1)], workspace=big))):
        with pytest.raises(pkv.PkvError) as e:
            fn()
        assert e.value.code == code
    assert pkv.launch_count() == n0


@pytest.mark.parametrize("bs,d", [(1, 64), (5, 32), (7, 128), (24, 64), (64, 32), (16, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 0), (30, 9), (200, 70)])
def test_f32_other_block_sizes(pkv, orc, bs, d, window, sinks):
    w = gen.decode_workload(seed=395 + bs, dtype="f32", num_q_heads=6, num_kv_heads=2, head_dim=d,
                            context_lens=[0, 3, 40, 333, 600], block_size=bs, window=window)
    if window:
        return check(pkv, orc, w, sinks)
    d_ = Dev(w)
    append(pkv, d_)
    out = call(pkv, w, d_, 0)
    torch.cuda.synchronize()
    kp, vp = w.k_pool.copy(), w.v_pool.copy()
    slots = pkv.slot_mapping_host(w.block_tables, w.num_blocks, w.new_rows, w.new_pos, bs)
    orc.append(kp, vp, "f32", slots, w.k_new, w.v_new)
    assert_close(to_f64(out), orc.decode(w.q, kp, vp, "f32", w.block_tables, w.seq_lens, 0, w.scale), "f32",
                 f"block size {bs}")
