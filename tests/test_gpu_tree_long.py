"""Drafted trees over long rows (GPU): every key is counted once, in every type and on
every kernel.  With queries of 0 every weight is 1 exactly, and with V rows of a single 1,
at dim p % D, an output is the share of its class among the attended keys (sums of ones
are exact in fp32; off by some steps of the quotient, 2^-22, and half a step of the output).
The elementwise bounds on random rows are wider than one key of some thousand where
weights are f16 (FP8 pools).

The loop of speculative steps again, over longer prompts, with the 2-norm of the latent outputs'
error beside their elementwise bounds: its two parts, the weights' and the output's
rounding, are 2^-8 each at most; one lost key of 400 would be 0.05."""
import numpy as np
import pytest
import torch

import test_gpu_tree_serving as serving
from tree_util import HALF, as_type, random_tree, seen, tables_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


@pytest.mark.parametrize("kind,hq,hkv,D,ctx,nodes,window", [
    ("bf16", 8, 8, 128, [20000, 700, 64], [4, 3, 2], 0), ("fp8", 16, 8, 128, [20000, 700, 64], [4, 3, 2], 0),
    ("bf16", 32, 8, 128, [12000, 3000, 65], [20, 1, 32], 0), ("fp8", 32, 8, 128, [12000, 3000, 65], [20, 1, 32], 0),
    ("bf16", 16, 4, 128, [9000, 5000, 100], [64, 1, 40], 0), ("fp8", 16, 4, 128, [9000, 5000, 100], [64, 1, 40], 0),
    ("bf16", 16, 4, 128, [2000] * 70, [1 + i % 64 for i in range(70)], 1500),
    ("fp8", 16, 4, 128, [2000] * 70, [1 + i % 64 for i in range(70)], 1500),
    ("bf16", 8, 2, 64, [6000, 90], [40, 9], 0), ("fp8", 8, 1, 256, [6000, 90], [40, 9], 0),
    ("f32", 4, 2, 64, [3000, 90], [20, 64], 0),
])
def test_every_key_counts_once(pkv, kind, hq, hkv, D, ctx, nodes, window):
    rng = np.random.RandomState(len(ctx) + D)
    C, lens = np.array(nodes), np.array(ctx) + np.array(nodes)
    cu = np.concatenate([[0], np.cumsum(C)]).astype(np.int32)
    masks = pkv.tree_masks_host(np.concatenate([random_tree(rng, c) for c in C]), cu)
    tables, nb = tables_for(rng, lens, np.maximum(0, np.array(ctx) - window + 1) if window else None)
    act = torch.float32 if kind == "f32" else torch.bfloat16
    if kind == "fp8":
        pools = pkv.fp8_pools(nb, hkv, D, "cuda")
    else:
        pools = [torch.full((nb, hkv, 16, D), float("nan"), dtype=act, device="cuda") for _ in range(2)]
    scales = dict(k_scale=1.0, v_scale=1.0) if kind == "fp8" else {}
    for r, L in enumerate(lens):
        p = np.array([x for x in range(int(L)) if tables[r, x // 16] >= 0])
        v = np.zeros((len(p), hkv, D))
        v[np.arange(len(p)), :, p % D] = 1
        slots = torch.from_numpy((tables[r, p // 16] * 16 + p % 16).astype(np.int32)).cuda()
        pkv.paged_kv_append(*pools, slots, as_type(np.ones_like(v), kind).cuda(), as_type(v, kind).cuda(), **scales)
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.paged_tree_attention(torch.zeros(int(cu[-1]), hq, D, dtype=act, device="cuda"), to(cu), to(masks), *pools,
                                   to(tables), to(lens.astype(np.int32)), int(C.max()), window, 0.1, status=status, **scales)
    assert int(status.item()) == 0
    out = out.double().cpu().numpy()
    for r, L in enumerate(lens):
        a, b = cu[r], cu[r + 1]
        ok = seen(int(L), int(C[r]), masks[a:b], window)
        want = np.stack([np.bincount(np.arange(int(L)) % D, weights=w, minlength=D) for w in ok]) / ok.sum(1, keepdims=True)
        err = np.abs(out[a:b] - want[:, None])
        assert (err <= (HALF[act] + 2.0 ** -22) * want[:, None]).all(), f"row {r}: {err.max()}"


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_speculative_steps_by_norm(pkv, kind, monkeypatch):
    plain, looked = serving.check, []

    def check(got, ref, mag, A, W, kind, dtype, what=""):
        plain(got, ref, mag, A, W, kind, dtype, what)
        if kind == "bf16 weights":
            err = np.linalg.norm(got.detach().double().cpu().numpy() - ref, axis=-1)
            assert (err <= 2.0 ** -7 * np.linalg.norm(ref, axis=-1)).all(), f"{what}: {err.max()}"
            looked.append(err.size)

    monkeypatch.setattr(serving, "check", check)
    with torch.cuda.stream(torch.cuda.Stream()):
        server = serving.Server(pkv, kind, 12)
        server.prompt([300, 33, 400])
        for nodes in ([3, 16, 4], [40, 1, 9], [4, 4, 4], [64, 17, 2]):
            server.step(nodes)
    assert sum(looked) > 1000
