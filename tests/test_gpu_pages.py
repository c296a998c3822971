"""Page copies (GPU): the pools after paged_copy_blocks equal numpy's byte for byte."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_paged_kv_gb300 as m
    return m


def make_pools(n, nb, hkv, bs, D, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    shape = (nb, hkv, bs * D) if dtype == torch.uint8 else (nb, hkv, bs, D)
    size = torch.empty(0, dtype=dtype).element_size()
    out = []
    for _ in range(2 * n):      # any bytes, NaN patterns among them
        b = torch.randint(0, 256, shape[:-1] + (shape[-1] * size,), generator=g, dtype=torch.uint8)
        out.append(b.cuda().view(dtype))
    return [(out[2 * i], out[2 * i + 1]) for i in range(n)]


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype,hkv,bs,D", [(torch.bfloat16, 8, 16, 128), (torch.bfloat16, 1, 16, 256),
                                            (torch.float32, 2, 16, 64), (torch.uint8, 8, 16, 128),
                                            (torch.bfloat16, 1, 1, 8), (torch.float32, 3, 5, 12),
                                            (torch.bfloat16, 7, 16, 72)])
@pytest.mark.parametrize("layers,n", [(1, 1), (3, 40), (70, 3)])
def test_copies_equal_numpy(pkv, dtype, hkv, bs, D, layers, n):
    nb = 2 * n + 3
    pools = make_pools(layers, nb, hkv, bs, D, dtype, seed=n)
    ids = np.random.default_rng(n).permutation(nb)
    src, dst = ids[:n], ids[n:2 * n]
    want = []
    for k, v in pools:
        for t in (k, v):
            a = raw(t).copy()
            a[dst] = a[src]
            want.append(a)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkv.check_block_copies(src, dst, nb)
    pkv.paged_copy_blocks(pkv.PoolSet(pools), i32(src), i32(dst), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    for a, t in zip(want, [t for kv in pools for t in kv]):
        assert np.array_equal(raw(t), a)


def test_one_source_many_destinations(pkv):
    pools = make_pools(1, 9000, 1, 16, 64, torch.bfloat16)
    a = raw(pools[0][0]).copy()
    dst = np.arange(1, 9000, dtype=np.int32)
    a[dst] = a[0]
    pkv.paged_copy_blocks(pkv.PoolSet(pools), i32(np.zeros_like(dst)), i32(dst))
    assert np.array_equal(raw(pools[0][0]), a)


def test_more_pairs_than_a_grid_dimension(pkv):
    n = 70000
    pools = make_pools(1, 2 * n, 1, 1, 8, torch.bfloat16)
    a = raw(pools[0][1]).copy()
    a[n:] = a[:n]
    pkv.paged_copy_blocks(pkv.PoolSet(pools), i32(np.arange(n)), i32(np.arange(n, 2 * n)))
    assert np.array_equal(raw(pools[0][1]), a)


def test_other_pools_of_another_size(pkv):
    old, new = make_pools(2, 10, 2, 16, 64, torch.bfloat16), make_pools(2, 25, 2, 16, 64, torch.bfloat16, seed=1)
    want = [raw(t).copy() for kv in new for t in kv]
    src, dst = [0, 9, 3], [24, 0, 3]
    for a, t in zip(want, [t for kv in old for t in kv]):
        a[dst] = raw(t)[src]
    pkv.paged_copy_blocks(pkv.PoolSet(old), i32(src), i32(dst), dst_pools=pkv.PoolSet(new))
    for a, t in zip(want, [t for kv in new for t in kv]):
        assert np.array_equal(raw(t), a)


def test_skipped_pairs_and_bad_ids(pkv):
    pools = make_pools(2, 8, 2, 16, 64, torch.bfloat16)
    want = [raw(t).copy() for kv in pools for t in kv]
    for a in want:
        a[5] = a[2]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    p = pkv.PoolSet(pools)
    pkv.paged_copy_blocks(p, i32([-1, 2, 3, 4]), i32([0, 5, -1, 4]), status=status)   # 4 -> 4 does nothing
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    pkv.paged_copy_blocks(p, i32([8, 1]), i32([0, 2 ** 31 - 1]), status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == pkv.DEV_BAD_BLOCK
    for a, t in zip(want, [t for kv in pools for t in kv]):
        assert np.array_equal(raw(t), a)


def test_far_blocks_past_32_bit_offsets(pkv):
    nb = (5 << 30) // (8 * 16 * 128 * 2)      # a pool over 4 GiB
    k = torch.zeros(nb, 8, 16, 128, dtype=torch.bfloat16, device="cuda")
    k[nb - 1] = 3
    k[1] = 5
    pkv.paged_copy_blocks(pkv.PoolSet([(k, k.clone())]), i32([nb - 1, 1]), i32([0, nb - 2]))
    assert bool((k[0] == 3).all()) and bool((k[nb - 2] == 5).all()) and bool((k[2] == 0).all())


def test_captured_and_replayed(pkv):
    pools = make_pools(2, 8, 2, 16, 64, torch.bfloat16)
    want = [raw(t).copy() for kv in pools for t in kv]
    for a in want:
        a[7] = a[1]
    p, src, dst = pkv.PoolSet(pools), i32([0]), i32([0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.paged_copy_blocks(p, src, dst)
    src.fill_(1)
    dst.fill_(7)
    g.replay()
    torch.cuda.synchronize()
    for a, t in zip(want, [t for kv in pools for t in kv]):
        assert np.array_equal(raw(t), a)


def test_refusals(pkv):
    pools = make_pools(1, 8, 2, 16, 64, torch.bfloat16)
    p = pkv.PoolSet(pools)
    n0 = pkv.launch_count()
    for src, dst in ((i32([1, 2]), i32([3])), (i32([1]).cpu(), i32([3])), (i32([1]).long(), i32([3])),
                     (i32([[1]]), i32([[3]]))):
        with pytest.raises(ValueError):
            pkv.paged_copy_blocks(p, src, dst)
    other = pkv.PoolSet(make_pools(1, 8, 2, 16, 128, torch.bfloat16))
    with pytest.raises(pkv.PkvError) as e:
        pkv.paged_copy_blocks(p, i32([1]), i32([2]), dst_pools=other)
    assert e.value.code == pkv.PKV_ERR_INVALID_ARG
    with pytest.raises(pkv.PkvError) as e:     # a page that is no whole number of 16-byte vectors
        pkv.paged_copy_blocks(pkv.PoolSet(make_pools(1, 8, 1, 1, 4, torch.bfloat16)), i32([1]), i32([2]))
    assert e.value.code == pkv.PKV_ERR_UNSUPPORTED
    pkv.paged_copy_blocks(p, i32([]), i32([]))
    assert pkv.launch_count() == n0
    with pytest.raises(ValueError):
        pkv.PoolSet([pools[0], make_pools(1, 8, 2, 16, 128, torch.bfloat16)[0]])
