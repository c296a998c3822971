"""Drafted trees and latent attention at many rows (GPU): more items than the levelled runs
look at, and workspaces sized once for the largest trees."""
import numpy as np
import pytest
import torch

from tree_util import attend, check, f64, seen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


def to(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def rows(pkv, B, C, most, seed):
    """B rows of up to `most` cached tokens and C drafts, pages in order: lengths, cu, masks, tables."""
    rng = np.random.RandomState(seed)
    n = rng.randint(0, most + 1, B)
    L = n + C
    pages = -(-L // 16)
    first = np.concatenate([[0], np.cumsum(pages)])
    tables = np.full((B, int(pages.max())), -1, dtype=np.int32)
    for b in range(tables.shape[1]):
        live = pages > b
        tables[live, b] = first[:-1][live] + b
    up = np.maximum(np.arange(C) - 1 - rng.randint(0, 3, (B, C)), -1)
    cu = (np.arange(B + 1) * C).astype(np.int32)
    return n, L.astype(np.int32), cu, pkv.tree_masks_host(up.reshape(-1), cu), tables, int(first[-1])


@pytest.mark.parametrize("kind,B,hq,hkv,C", [("bf16", 8300, 16, 8, 9), ("bf16", 8300, 32, 8, 33), ("fp8", 8300, 16, 8, 9),
                                             ("bf16", 9000, 8, 8, 2)])
def test_trees_of_many_rows(pkv, kind, B, hq, hkv, C):
    n, L, cu, masks, tables, nb = rows(pkv, B, C, 40, 1)
    D, g = 128, torch.Generator(device="cuda").manual_seed(2)
    if kind == "fp8":
        pools = [(torch.randn(nb, hkv, 16 * D, generator=g, device="cuda") / 0.02).clamp(-448, 448)
                 .to(torch.float8_e4m3fn).view(torch.uint8) for _ in range(2)]
    else:
        pools = [torch.randn(nb, hkv, 16, D, generator=g, device="cuda").bfloat16() for _ in range(2)]
    q = torch.randn(B * C, hq, D, generator=g, device="cuda").bfloat16()
    scales = dict(k_scale=0.02, v_scale=0.02) if kind == "fp8" else {}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, float("nan"))
    args = [to(cu), to(masks), *pools]
    pkv.paged_tree_attention(q, *args, to(tables), to(L), C, 0, 0.1, out=out, status=status, **scales)
    assert int(status.item()) == 0 and torch.isfinite(out).all()
    # the same rows in calls of some hundred: the elementwise bound's two sides of each
    for a in range(0, B, 700):
        b = min(B, a + 700)
        part = pkv.paged_tree_attention(q[a * C:b * C], to(cu[:b - a + 1]), args[1][a * C:b * C], *pools, to(tables[a:b]), to(L[a:b]),
                                        C, 0, 0.1, **scales)
        diff = (part.float() - out[a * C:b * C].float()).abs()
        # both are within half a step of the exact value and 2^-10 (FP8; 2^-16) of the weighted magnitudes, which 6 bounds
        # (the largest of N(0, 1) values here is below it)
        assert (diff <= 2.0 ** -7 * 1.01 * part.float().abs() + (2.0 ** -9 if kind == "fp8" else 2.0 ** -15) * 6).all()
    if kind == "bf16":
        for r in (0, 1, B // 2, B - 1):
            pages = to(tables[r, :-(-int(L[r]) // 16)]).long()
            k, v = [f64(p[pages].transpose(1, 2).reshape(-1, hkv, D)[:int(L[r])]) for p in pools]
            ok = seen(int(L[r]), C, masks[cu[r]:cu[r + 1]])
            for h in range(0, hq, 5):
                ref, mag, A = attend(f64(q[r * C:(r + 1) * C, h]), k[:, h * hkv // hq], v[:, h * hkv // hq], ok, 0.1)
                check(out[r * C:(r + 1) * C, h], ref, mag, A, D, kind, torch.bfloat16, f"row {r} head {h}")


def test_latent_of_many_rows(pkv):
    B, C, H, R, Dr = 20000, 3, 48, 256, 64
    n, L, cu, masks, tables, nb = rows(pkv, B, C, 40, 3)
    g = torch.Generator(device="cuda").manual_seed(2)
    pool = torch.randn(nb, 16, R + Dr, generator=g, device="cuda").bfloat16()
    q = (torch.randn(B * C, H, R + Dr, generator=g, device="cuda") * 0.2).bfloat16()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = pkv.paged_latent_attention(q, pool, R, to(tables), to(L), 0.125, cu_q_lens=to(cu), max_q_len=C, tree_masks=to(masks),
                                     status=status)
    assert int(status.item()) == 0 and torch.isfinite(out).all()
    for r in (0, 1, 777, B // 2, B - 1):
        rows_ = f64(pool[to(tables[r, :-(-int(L[r]) // 16)]).long()].reshape(-1, R + Dr)[:int(L[r])])
        ok = seen(int(L[r]), C, masks[cu[r]:cu[r + 1]])
        for h in range(0, H, 7):
            ref, mag, A = attend(f64(q[r * C:(r + 1) * C, h]), rows_, rows_[:, :R], ok, 0.125)
            check(out[r * C:(r + 1) * C, h], ref, mag, A, R + Dr, "bf16 weights", torch.bfloat16, f"row {r} head {h}")


@pytest.mark.parametrize("hq,hkv,D", [(32, 8, 128), (16, 8, 128), (12, 4, 128), (8, 1, 256), (8, 8, 64), (16, 1, 128)])
def test_workspace_of_the_largest_tree_holds_every_smaller_one(pkv, hq, hkv, D):
    rng = np.random.RandomState(hq + D)
    for _ in range(40):
        batch, most, window = int(2 ** rng.uniform(0, 13)), int(2 ** rng.uniform(4, 16)), int(rng.choice([0, 64, 5000]))
        size = [pkv.tree_workspace_size(batch, hq, hkv, D, 16, n, most, window) for n in range(1, 65)]
        assert size == sorted(size) and size[0] > 0
        assert pkv.tree_workspace_size(batch, hq, hkv, D, 16, 64, max(1, most // 3), window) <= size[-1]


def test_a_smaller_step_in_the_largest_workspace(pkv):
    B, hq, hkv, D = 800, 32, 8, 128
    n, L, cu, masks, tables, nb = rows(pkv, B, 4, 400, 5)
    pools = [torch.randn(nb, hkv, 16, D, device="cuda").bfloat16() for _ in range(2)]
    q = torch.randn(B * 4, hq, D, device="cuda").bfloat16()
    ws = pkv.alloc_workspace(pkv.tree_workspace_size(B, hq, hkv, D, 16, 64, 512), "cuda")
    out = pkv.paged_tree_attention(q, to(cu), to(masks), *pools, to(tables), to(L), 4, 0, 0.1, workspace=ws, max_seq_len=512)
    assert torch.equal(out, pkv.paged_tree_attention(q, to(cu), to(masks), *pools, to(tables), to(L), 4, 0, 0.1, max_seq_len=512))
