"""The workspace a size query reports holds every call of that length or a
shorter one: a plan's splits grow in steps, so a shorter length can need more."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


def need(pkv, rows, batch, hq, hkv, d, bs, blocks):
    """Bytes a plan over `blocks` blocks a row takes: per (row, q head, split) d
    floats, then two."""
    splits = pkv.decode_plan(batch, hq, hkv, d, bs, blocks * bs)[0]
    n = rows * hq * splits * 4
    return (n * d + 255) // 256 * 256 + 2 * n


def shorter(rng, n):
    return sorted({1, n} | {max(1, n - k) for k in range(40)} | {int(x) for x in rng.integers(1, n + 1, 60)})


@pytest.mark.parametrize("seed", range(6))
def test_decode_and_verify_sizes_hold_for_every_shorter_length(pkv, seed):
    rng = np.random.default_rng(seed)
    for _ in range(25):
        batch, hkv, g = int(rng.integers(1, 65)), int(rng.choice([1, 2, 4, 8])), int(rng.choice([1, 4, 8]))
        d, bs, hq = int(rng.choice([64, 128, 256])), 16, hkv * g
        n = int(2 ** rng.uniform(2, 13))
        size = pkv.decode_workspace_size(batch, hq, hkv, d, bs, n * bs)
        assert all(size >= need(pkv, batch, batch, hq, hkv, d, bs, k) for k in shorter(rng, n))
        if g <= 4:          # a verify step: 16 / g queries a row
            size = pkv.prefill_workspace_size(batch, hq, hkv, d, bs, 16 // g, n * bs)
            assert all(size >= need(pkv, batch * 16 // g, batch, hq, hkv, d, bs, k) for k in shorter(rng, n))
        # a window with sinks: at most their blocks and one more
        window, sinks = int(rng.integers(1, n * bs)), int(rng.integers(1, 100))
        size = pkv.decode_workspace_size(batch, hq, hkv, d, bs, n * bs, window, sinks=sinks)
        most = min(n, -(-window // bs) + 1 + -(-sinks // bs))
        assert all(size >= need(pkv, batch, batch, hq, hkv, d, bs, k) for k in shorter(rng, most))


@pytest.mark.parametrize("batch,hkv", [(1, 1), (4, 1), (32, 4), (64, 8)])
def test_sizes_grow_with_the_length(pkv, batch, hkv):
    for size in (lambda n: pkv.decode_workspace_size(batch, 4 * hkv, hkv, 128, 16, n),
                 lambda n: pkv.decode_workspace_size(batch, 4 * hkv, hkv, 128, 16, n, 5000, sinks=4),
                 lambda n: pkv.prefill_workspace_size(batch, 4 * hkv, hkv, 128, 16, 4, n),
                 lambda n: pkv.prefill_workspace_size(batch, 4 * hkv, hkv, 128, 16, 20, n)):
        sizes = [size(n) for n in range(1, 40000, 61)]
        assert sizes == sorted(sizes)


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (20000, 0), (20000, 4)])
def test_a_bound_past_the_tables_is_served(pkv, window, sinks):
    # tables of 304 blocks, max_seq_len 65536: the call plans for the tables,
    # with more splits than a plan for 65536 tokens has
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    B, blocks, D = 4, 304, 128
    gen = torch.Generator("cuda").manual_seed(3)
    kp, vp = (torch.randn(B * blocks, 1, 16, D, generator=gen, device="cuda").bfloat16() for _ in range(2))
    tables = torch.randperm(B * blocks, generator=gen, device="cuda").int().view(B, blocks)
    lens = torch.tensor([4864, 4001, 17, 2500], dtype=torch.int32, device="cuda")
    scale = D ** -0.5
    q = torch.randn(B, 4, D, generator=gen, device="cuda").bfloat16()
    kw = dict(sinks=sinks) if sinks else {}
    want = pkv.paged_decode_attention(q, kp, vp, tables, lens, window, scale, max_seq_len=4864, **kw)
    got = pkv.paged_decode_attention(q, kp, vp, tables, lens, window, scale, max_seq_len=65536, **kw)
    assert torch.equal(got, want)
    ws = pkv.alloc_workspace(pkv.decode_workspace_size(B, 4, 1, D, 16, 65536, window, sinks=sinks), "cuda")
    for n in (4864, 5000, 10000, 30000):        # one workspace, shorter calls
        assert torch.equal(pkv.paged_decode_attention(q, kp, vp, tables, lens, window, scale, max_seq_len=n,
                                                      workspace=ws, **kw), want)
    groups = [pkv.DecodeGroup(q, kp, vp, tables, lens, window, scale, max_seq_len=65536, sinks=sinks)
              for _ in range(2)]
    for got in pkv.paged_decode_attention_groups(groups):
        assert torch.equal(got, want)
    q4 = torch.randn(B * 4, 4, D, generator=gen, device="cuda").bfloat16()
    cu = torch.arange(0, 4 * B + 1, 4, dtype=torch.int32, device="cuda")
    a = (q4, cu, kp, vp, tables, lens, 4, window, scale)
    assert torch.equal(pkv.paged_prefill_chunk_attention(*a, max_seq_len=65536, **kw),
                       pkv.paged_prefill_chunk_attention(*a, max_seq_len=4864, **kw))
