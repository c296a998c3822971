"""Measured cases of the paged cache's operators around a serving step.

Three operators, each in a plain form (elementary torch operations) and, where
``own`` is true, as the calls a user makes of the library:

- ``rope``: rotary positions (one or three axes) applied to q and k, the
  rotated K rows and the V rows written into their pool slots;
- ``sinks_decode`` / ``sinks_prefill``: paged attention with a sliding window
  whose first ``sinks`` positions stay visible, one query per row or a chunk;
- ``copy``: pages of every layer's K and V pool copied to other pages (fork,
  compaction).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a decode step of 32 requests (32 q / 8 kv heads): every call is this small while tokens stream
        dict(name="rope_step_b32", op="rope", dtype="bf16", tokens=32, hq=32, hkv=8, dim=128,
             rotary=128, axes=1, interleaved=False, far=131072),
        # a prefill step of 4 chunks of 512 with image tokens: time, height and width axes
        dict(name="rope_chunk_2048_3axes", op="rope", dtype="bf16", tokens=2048, hq=32, hkv=8,
             dim=128, rotary=128, axes=3, interleaved=False, far=32768),
        # the small f32 model's prompt, an odd length, half of the head rotated in adjacent pairs, far positions
        dict(name="rope_odd_777_f32", op="rope", dtype="f32", tokens=777, hq=4, hkv=2, dim=64,
             rotary=32, axes=1, interleaved=True, far=4000000),
        # a whole context into an FP8 cache
        dict(name="rope_context_16384_fp8", op="rope", dtype="fp8", tokens=16384, hq=32, hkv=8,
             dim=128, rotary=128, axes=3, interleaved=False, far=131072),
        # a few long streams over a window of 512: latency counts
        dict(name="sinks_decode_b4_w512_d256", op="sinks_decode", dtype="bf16", batch=4, hq=8,
             hkv=1, dim=256, window=512, sinks=4, ctx_min=32768, ctx_max=32768),
        # a batch whose rows are shorter and longer than the window
        dict(name="sinks_decode_b32_w4096", op="sinks_decode", dtype="bf16", batch=32, hq=32, hkv=8,
             dim=128, window=4096, sinks=4, ctx_min=1024, ctx_max=8192),
        # endless streams on an FP8 cache, far past any trained length
        dict(name="sinks_decode_b64_w2048_fp8", op="sinks_decode", dtype="fp8", batch=64, hq=32,
             hkv=8, dim=128, window=2048, sinks=16, ctx_min=100000, ctx_max=1000000),
        # the chunked-prefill step over a window
        dict(name="sinks_prefill_4x512_w4096", op="sinks_prefill", dtype="bf16", batch=4, hq=32,
             hkv=8, dim=128, window=4096, sinks=4, prefix_min=16384, prefix_max=16384,
             chunk_min=512, chunk_max=512),
        # ragged prompts on an FP8 cache, odd window, sinks that end inside a page
        dict(name="sinks_prefill_ragged_fp8", op="sinks_prefill", dtype="fp8", batch=8, hq=16,
             hkv=4, dim=128, window=1000, sinks=5, prefix_min=0, prefix_max=3000,
             chunk_min=1, chunk_max=700),
        # long prompts in one chunk each
        dict(name="sinks_prefill_2x4096_w4096", op="sinks_prefill", dtype="bf16", batch=2, hq=32,
             hkv=8, dim=128, window=4096, sinks=64, prefix_min=0, prefix_max=4096,
             chunk_min=4096, chunk_max=4096),
        # a fork of 32 requests: one partial page each, 4 layers
        dict(name="copy_fork_32x4", op="copy", dtype="bf16", layers=4, pages=512, moves=32, hkv=8,
             dim=128),
        # compaction of a grown pool
        dict(name="copy_compact_4096x2", op="copy", dtype="bf16", layers=2, pages=8200, moves=4096,
             hkv=8, dim=128),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = [(32, 8, 128), (16, 8, 128), (8, 1, 256), (16, 4, 128), (6, 2, 64)]


def draw(rng):
    op = rng.choice(["rope", "rope", "sinks_decode", "sinks_decode", "sinks_prefill", "copy"])
    dtype = rng.choice(["bf16", "bf16", "fp8"])
    hq, hkv, dim = rng.choice(_HEADS)
    if op == "rope":
        if rng.random() < 0.2:
            dtype, hq, hkv, dim = "f32", 4, 2, 64
        axes = rng.choice([1, 3])
        return dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, 16384), hq=hq, hkv=hkv, dim=dim,
                    rotary=dim if rng.random() < 0.7 else dim // 2, axes=axes,
                    interleaved=rng.random() < 0.3, far=_log_int(rng, 1000, 4000000))
    if op == "sinks_decode":
        window = _log_int(rng, 64, 4096)
        if rng.random() < 0.15:
            dtype, hq, hkv, dim = "f32", 4, 2, 64
        lo = _log_int(rng, 1, 100000)
        return dict(op=op, dtype=dtype, batch=_log_int(rng, 1, 64), hq=hq, hkv=hkv, dim=dim,
                    window=window, sinks=rng.choice([1, 4, 5, 16, 64, 100]), ctx_min=lo,
                    ctx_max=lo + _log_int(rng, 1, 100000))
    if op == "sinks_prefill":
        hq, hkv, dim = rng.choice([(32, 8, 128), (16, 8, 128), (16, 4, 128)])
        top = _log_int(rng, 2, 1024)
        return dict(op=op, dtype=dtype, batch=_log_int(rng, 1, 8), hq=hq, hkv=hkv, dim=dim,
                    window=_log_int(rng, 64, 4096), sinks=rng.choice([1, 4, 5, 16, 64, 100]),
                    prefix_min=0, prefix_max=_log_int(rng, 1, 20000),
                    chunk_min=rng.choice([1, top]), chunk_max=top)
    moves = _log_int(rng, 1, 4096)
    return dict(op=op, dtype=dtype, layers=rng.choice([1, 2, 5]) if moves < 1500 else 1,
                pages=2 * moves + rng.randint(1, 600), moves=moves, hkv=hkv, dim=dim)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
DEV = "cuda"
K_SCALE, V_SCALE = float(np.float32(0.0123)), float(np.float32(0.0171))
_ACT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.bfloat16}


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(DEV)


def _tile_order(dim):
    """Byte of (token, dim) in an FP8 tile, K and V: int64 [16, dim] each."""
    t = torch.arange(BLOCK, device=DEV)[:, None]
    d = torch.arange(dim, device=DEV)[None, :]
    k = d % 16
    kb = (d // 64) * 1024 + (t // 8) * 512 + ((t % 8) * 4 + (k % 8) // 2) * 16 + ((d % 64) // 16) * 4 \
        + k % 2 + 2 * (k // 8)
    vb = (d // 32) * 512 + ((d % 8) * 4 + (t % 8) // 2) * 16 + ((d % 32) // 8) * 4 + t % 2 + 2 * (t // 8)
    return kb, vb


def _pools(g, nb, hkv, dim, dtype):
    """K and V pools full of N(0, 1) values (FP8: codes of N(0, 1) / scale)."""
    if dtype != "fp8":
        return [_normal(g, (nb, hkv, BLOCK, dim), _ACT[dtype]) for _ in range(2)]
    return [(_normal(g, (nb, hkv, BLOCK * dim), torch.float32) / s).clamp(-448, 448)
            .to(torch.float8_e4m3fn).view(torch.uint8) for s in (K_SCALE, V_SCALE)]


def _inv_freq(rotary):
    return 10000.0 ** (-2.0 * np.arange(rotary // 2, dtype=np.float64) / rotary)


def _axis_of_pair(rotary, axes):
    """Runs of the pairs: a quarter for time, the rest for height and width."""
    n = rotary // 2
    if axes == 1:
        return np.zeros(n, dtype=np.int64)
    first = n // 4
    second = first + (n - first) // 2
    return np.where(np.arange(n) < first, 0, np.where(np.arange(n) < second, 1, 2))


def _lengths(case):
    """Tokens and queries of each row: drawn once for a case, whatever the seed."""
    B, spread = case["batch"], np.random.RandomState(case["batch"] * 65537 + case["window"])
    if case["op"] == "sinks_decode":
        return spread.randint(case["ctx_min"], case["ctx_max"] + 1, B), np.ones(B, dtype=np.int64)
    prefix = spread.randint(case["prefix_min"], case["prefix_max"] + 1, B)
    chunks = spread.randint(case["chunk_min"], case["chunk_max"] + 1, B)
    chunks[0] = case["chunk_max"]
    return prefix + chunks, chunks


def _live_tables(rng, lens, lo, sinks, width):
    """Block tables of rows that hold their sink pages and the pages from position lo on."""
    tables = np.full((len(lens), width), -1, dtype=np.int64)
    held = np.zeros((len(lens), width), dtype=bool)
    for r, n in enumerate(lens):
        end = -(-int(n) // BLOCK)
        held[r, int(lo[r]) // BLOCK:end] = True
        held[r, :min(end, -(-sinks // BLOCK))] = True
    count = int(held.sum())
    nb = max(count, 1)
    tables[held] = rng.permutation(nb)[:count]
    return tables, nb


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rng = np.random.RandomState(seed % (1 << 32))
    s = dict(case)
    op, dtype = case["op"], case["dtype"]
    act = _ACT[dtype]
    if op == "copy":
        shape = (case["layers"], 2, case["pages"], case["hkv"], BLOCK, case["dim"])
        if dtype == "fp8":
            shape = shape[:4] + (BLOCK * case["dim"],)
            s["cache"] = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
        else:
            s["cache"] = _normal(g, shape, act)
        ids = rng.permutation(case["pages"])
        s["src"], s["dst"] = _i32(ids[:case["moves"]]), _i32(ids[case["moves"]:2 * case["moves"]])
        s["src64"], s["dst64"] = s["src"].long(), s["dst"].long()
        if own:
            import block_paged_kv_gb300 as pkv
            s["pools"] = pkv.PoolSet([(s["cache"][i, 0], s["cache"][i, 1]) for i in range(case["layers"])])
        return s
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    if op == "rope":
        T, rd, axes = case["tokens"], case["rotary"], case["axes"]
        nb = -(-T // BLOCK) + 64
        s["k_pool"], s["v_pool"] = _pools(g, nb, hkv, dim, dtype)
        # rows cut from one projection's output, as a model has them
        qkv = _normal(g, (T, (hq + 2 * hkv) * dim), act)
        s["q"] = qkv[:, :hq * dim].view(T, hq, dim)
        s["k"] = qkv[:, hq * dim:(hq + hkv) * dim].view(T, hkv, dim)
        s["v"] = qkv[:, (hq + hkv) * dim:].view(T, hkv, dim)
        if T <= 64:   # a decode step: one token per request, anywhere in its page
            slots = rng.permutation(nb)[:T] * BLOCK + rng.randint(0, BLOCK, T)
            pos = rng.randint(0, case["far"], T)[None].repeat(axes, 0)
        else:         # a run of tokens through shuffled pages, starting inside one
            start = int(rng.randint(0, BLOCK))
            at = start + np.arange(T)
            slots = rng.permutation(nb)[at // BLOCK] * BLOCK + at % BLOCK
            pos = (rng.randint(0, case["far"]) + np.arange(T))[None].repeat(axes, 0)
        if axes == 3:  # an image of up to 64 columns: height and width of each token within it
            cols = int(rng.randint(8, 65))
            base = pos[0] - np.arange(T) * (T > 64)
            pos[1], pos[2] = base + np.arange(T) // cols, base + np.arange(T) % cols
        s["slots"], s["pos"] = _i32(slots), _i32(pos)
        s["inv_freq"] = torch.from_numpy(_inv_freq(rd)).to(DEV)
        s["axis"] = torch.from_numpy(_axis_of_pair(rd, axes)).to(DEV)
        s["blk"], s["off"] = s["slots"].long() // BLOCK, s["slots"].long() % BLOCK
        s["q_out"] = torch.empty((T, hq, dim), dtype=act, device=DEV)
        if dtype == "fp8":
            s["k_order"], s["v_order"] = _tile_order(dim)
        if own:
            import block_paged_kv_gb300 as pkv
            s["rope"] = pkv.make_rope(_inv_freq(rd), axis_of_pair=_axis_of_pair(rd, axes),
                                      interleaved=case["interleaved"])
        return s
    B, W, S = case["batch"], case["window"], case["sinks"]
    lens, chunks = _lengths(case)
    lo = np.maximum(0, lens - chunks + 1 - W)
    width = -(-int(lens.max()) // BLOCK)
    tables, nb = _live_tables(rng, lens, lo, S, width)
    s["k_pool"], s["v_pool"] = _pools(g, nb, hkv, dim, dtype)
    s["tables"], s["lens"] = _i32(tables), _i32(lens)
    s["scale"] = 1.0 / math.sqrt(dim)
    s["max_len"], s["max_q"] = int(lens.max()), int(chunks.max())
    s["q"] = _normal(g, (int(chunks.sum()), hq, dim), act)
    s["cu"] = _i32(np.concatenate([[0], np.cumsum(chunks)]))
    s["out"] = torch.empty_like(s["q"])
    if dtype == "fp8":
        s["k_order"], s["v_order"] = _tile_order(dim)
    if own:
        import block_paged_kv_gb300 as pkv
        if op == "sinks_decode":
            need = pkv.decode_workspace_size(B, hq, hkv, dim, BLOCK, s["max_len"], W, sinks=S)
        else:
            need = pkv.prefill_workspace_size(B, hq, hkv, dim, BLOCK, s["max_q"], s["max_len"], W, sinks=S)
        s["workspace"] = pkv.alloc_workspace(need, DEV)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rotate(x, cos, sin, rotary, interleaved):
    """x [T, H, D] (f32) with its first `rotary` dims rotated; cos, sin [T, rotary / 2]."""
    y = x.clone()
    cos, sin = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rotary:2], x[..., 1:rotary:2]
        y[..., 0:rotary:2], y[..., 1:rotary:2] = a * cos - b * sin, b * cos + a * sin
    else:
        h = rotary // 2
        a, b = x[..., :h], x[..., h:rotary]
        y[..., :h], y[..., h:rotary] = a * cos - b * sin, b * cos + a * sin
    return y


def _plain_rope(s):
    rd, inter = s["rotary"], s["interleaved"]
    angle = s["pos"].double()[s["axis"]].t() * s["inv_freq"]  # [T, rd / 2]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    act = s["q"].dtype
    q = _rotate(s["q"].float(), cos, sin, rd, inter).to(act)
    k, v = _rotate(s["k"].float(), cos, sin, rd, inter), s["v"]
    kp, vp = s["k_pool"], s["v_pool"]
    if s["dtype"] == "fp8":
        kc = (k / K_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        vc = (v.float() / V_SCALE).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        heads = torch.arange(s["hkv"], device=DEV)
        at = (s["blk"][:, None, None], heads[None, :, None])
        kp[at + (s["k_order"][s["off"]][:, None, :],)] = kc
        vp[at + (s["v_order"][s["off"]][:, None, :],)] = vc
        return q, kp.view(torch.float8_e4m3fn), vp.view(torch.float8_e4m3fn)
    kp[s["blk"], :, s["off"]] = k.to(act)
    vp[s["blk"], :, s["off"]] = v
    return q, kp, vp


def _rows(s, pool, order, scale, blk, off):
    """Pool rows at (blk, off) [B, n] as f32 [B, n, Hkv, D]."""
    if s["dtype"] != "fp8":
        return pool[blk, :, off].float()
    values = pool.view(torch.float8_e4m3fn).float() * scale
    return values[:, :, order][blk, :, off]


def _plain_attention(s):
    B, W, S = s["batch"], s["window"], s["sinks"]
    hq, hkv, dim = s["hq"], s["hkv"], s["dim"]
    C, T = s["max_q"], s["q"].shape[0]
    cu, L = s["cu"].long(), s["lens"].long()
    n_q = cu[1:] - cu[:-1]
    first = L - n_q                                     # position of a row's first query
    lo = (first - W + 1).clamp(min=0)                   # where its window starts
    sink = torch.arange(S, device=DEV).expand(B, S)
    win = lo[:, None] + torch.arange(W + C - 1, device=DEV)
    pos = torch.cat([sink, win], 1)                     # [B, n]
    real = torch.cat([sink < lo[:, None], win < L[:, None]], 1)
    pos = torch.where(real, pos, 0)
    blk = s["tables"].long().gather(1, pos // BLOCK).clamp(min=0)
    k = _rows(s, s["k_pool"], s.get("k_order"), K_SCALE, blk, pos % BLOCK)
    v = _rows(s, s["v_pool"], s.get("v_order"), V_SCALE, blk, pos % BLOCK)
    at = torch.arange(C, device=DEV)
    q = s["q"][(cu[:-1, None] + at).clamp(max=T - 1)].float()                       # [B, C, Hq, D]
    q = q.view(B, C, hkv, hq // hkv, dim).permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, dim)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                     # [B, Hkv, G * C, n]
    score = score.view(B, hkv, hq // hkv, C, -1)
    qpos = (first[:, None] + at)[:, :, None]                                        # [B, C, 1]
    seen = real[:, None] & (pos[:, None] <= qpos) & ((pos[:, None] > qpos - W) | (pos[:, None] < S))
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-1e30))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    o = torch.matmul(p.view(B, hkv, -1, p.shape[-1]), v.permute(0, 2, 1, 3))
    o = o.view(B, hq, C, dim).transpose(1, 2).to(s["q"].dtype)                      # [B, C, Hq, D]
    i = torch.arange(T, device=DEV)
    row = torch.bucketize(i, cu[1:], right=True)
    return o[row, i - cu[row]]


def _plain_copy(s):
    cache = s["cache"]
    cache[:, :, s["dst64"]] = cache[:, :, s["src64"]]
    return cache


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------
def _own_rope(pkv, s):
    pkv.paged_kv_append_rope(s["k_pool"], s["v_pool"], s["slots"], s["q"], s["k"], s["v"], s["pos"],
                             s["rope"], q_out=s["q_out"], k_scale=K_SCALE, v_scale=V_SCALE)
    if s["dtype"] == "fp8":
        return s["q_out"], s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn)
    return s["q_out"], s["k_pool"], s["v_pool"]


def _own_attention(pkv, s):
    if s["op"] == "sinks_decode":
        return pkv.paged_decode_attention(s["q"], s["k_pool"], s["v_pool"], s["tables"], s["lens"],
                                          s["window"], s["scale"], out=s["out"],
                                          workspace=s["workspace"], max_seq_len=s["max_len"],
                                          k_scale=K_SCALE, v_scale=V_SCALE, sinks=s["sinks"])
    return pkv.paged_prefill_chunk_attention(s["q"], s["cu"], s["k_pool"], s["v_pool"], s["tables"],
                                             s["lens"], s["max_q"], s["window"], s["scale"],
                                             out=s["out"], workspace=s["workspace"],
                                             max_seq_len=s["max_len"], k_scale=K_SCALE,
                                             v_scale=V_SCALE, sinks=s["sinks"])


def run(s):
    if own:
        import block_paged_kv_gb300 as pkv
        if s["op"] == "rope":
            return _own_rope(pkv, s)
        if s["op"] == "copy":
            pkv.paged_copy_blocks(s["pools"], s["src"], s["dst"])
            return s["cache"]
        return _own_attention(pkv, s)
    if s["op"] == "rope":
        return _plain_rope(s)
    if s["op"] == "copy":
        return _plain_copy(s)
    return _plain_attention(s)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    op = case["op"]
    elem = {"f32": 4, "bf16": 2, "fp8": 1}[case["dtype"]]
    act = 4 if case["dtype"] == "f32" else 2
    if op == "copy":
        n = case["layers"] * 2 * case["moves"] * case["hkv"] * BLOCK * case["dim"] * elem
        return {"bytes": 2 * n + 8 * case["moves"], "flops": 0}
    hq, hkv, dim = case["hq"], case["hkv"], case["dim"]
    if op == "rope":
        T = case["tokens"]
        row = 2 * hq * dim * act + 2 * hkv * dim * (act + elem) + 4 + 4 * case["axes"]
        return {"bytes": T * row + 4 * case["rotary"], "flops": T * (hq + hkv) * case["rotary"] * 3}
    W, S = case["window"], case["sinks"]
    lens, chunks = _lengths(case)
    first = lens - chunks                       # position of a row's first query
    lo = np.maximum(0, first - W + 1)           # where its window starts
    seen = int((lens - lo + np.minimum(S, lo)).sum())
    pairs = 0
    for p, c in zip(first, chunks):
        at = np.arange(p, p + c)
        pairs += int(np.minimum(at + 1, W + np.minimum(S, np.maximum(0, at - W + 1))).sum())
    return {"bytes": seen * 2 * hkv * dim * elem + 2 * int(chunks.sum()) * hq * dim * act + seen // BLOCK * 4,
            "flops": 4 * dim * hq * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    if case["op"] == "copy":
        return None  # nothing is computed
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s)
    if s["batch"] * s["hq"] * s["max_q"] * (s["window"] + s["sinks"] + s["max_q"]) > 3e9:
        return None
    return _exact_attention(s)


def _exact_rope(s):
    rd = s["rotary"]
    n = rd // 2
    pos = s["pos"].cpu().numpy().astype(np.longdouble)
    freq = s["inv_freq"].cpu().numpy().astype(np.longdouble)
    axis = s["axis"].cpu().numpy()
    angle = np.stack([pos[axis[i]] * freq[i] for i in range(n)], 1)
    turn = torch.from_numpy(np.exp(1j * np.fmod(angle, 2 * np.longdouble(np.pi)).astype(np.float64))).to(DEV)

    def rotated(x):
        x = x.double()
        head, rest = x[..., :rd], x[..., rd:]
        pair = head.unflatten(-1, (n, 2)) if s["interleaved"] else head.unflatten(-1, (2, n)).transpose(-1, -2)
        z = torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous()) * turn[:, None]
        out = torch.stack([z.real, z.imag], -1 if s["interleaved"] else -2).flatten(-2)
        return torch.cat([out, rest], -1)

    q, k, v = rotated(s["q"]), rotated(s["k"]), s["v"].double()
    if s["dtype"] != "fp8":
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
        for pool, rows in ((kp, k), (vp, v)):
            by_slot = pool.transpose(1, 2).clone(memory_format=torch.contiguous_format)
            by_slot.view(-1, s["hkv"], s["dim"])[s["slots"].long()] = rows
            pool.copy_(by_slot.transpose(1, 2))
        return q, kp, vp
    out = []
    for pool, rows, scale, order in ((s["k_pool"], k, K_SCALE, s["k_order"]), (s["v_pool"], v, V_SCALE, s["v_order"])):
        values = pool.view(torch.float8_e4m3fn).double().flatten()
        tile = BLOCK * s["dim"]
        base = (s["blk"][:, None] * s["hkv"] + torch.arange(s["hkv"], device=DEV)) * tile
        values[base[:, :, None] + order[s["off"]][:, None, :]] = (rows / scale).clamp(-448, 448)
        out.append(values.view(pool.shape))
    return q, out[0], out[1]


def _exact_attention(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    cu, lens = s["cu"].tolist(), s["lens"].tolist()
    G = s["hq"] // s["hkv"]
    for r, L in enumerate(lens):
        first = L - (cu[r + 1] - cu[r])
        keys = torch.arange(L, device=DEV)
        keys = keys[(keys < s["sinks"]) | (keys > first - s["window"])]
        blk = s["tables"][r].long()[keys // BLOCK]
        side = []
        for name, scale in (("k", K_SCALE), ("v", V_SCALE)):
            pool = s[name + "_pool"][blk]               # [n, Hkv, 16, D] or tile bytes
            if s["dtype"] == "fp8":
                pool = (pool.view(torch.float8_e4m3fn).double() * scale)[:, :, s[name + "_order"]]
            side.append(pool[torch.arange(len(keys), device=DEV), :, keys % BLOCK].double())
        at = torch.arange(first, L, device=DEV)[:, None]
        hidden = (keys > at) | ((keys >= s["sinks"]) & (keys <= at - s["window"]))
        for h in range(s["hq"]):
            score = s["q"][cu[r]:cu[r + 1], h].double() @ side[0][:, h // G].t() * s["scale"]
            weight = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
            out[cu[r]:cu[r + 1], h] = weight @ side[1][:, h // G]
    return out
