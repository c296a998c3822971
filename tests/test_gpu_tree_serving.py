"""Drafted trees as a server runs them: reserve pages, append the drafts, attend, accept
a path, commit it, give the other pages back; a K/V cache and a latent cache that
share block ids, two layers each, on one stream and one workspace."""
import numpy as np
import pytest
import torch

from tree_util import as_type, attend, check, f64, random_tree, seen

pytestmark = pytest.mark.gpu

LAYERS, BS, HQ, HKV, D, H, R, DR, NB = 2, 16, 16, 4, 128, 16, 256, 64, 64
KS, VS = 0.0123, 0.0171


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


def to(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Server:
    def __init__(self, pkv, kind, seed):
        self.pkv, self.kind, self.rng = pkv, kind, np.random.RandomState(seed)
        self.alloc = pkv.BlockAllocator(BS, 4, NB)
        self.req = [self.alloc.begin() for _ in range(3)]
        if kind == "fp8":
            self.kv = [pkv.fp8_pools(NB, HKV, D, "cuda") for _ in range(LAYERS)]
        else:
            self.kv = [tuple(torch.full((NB, HKV, BS, D), float("nan"), device="cuda").bfloat16() for _ in range(2))
                       for _ in range(LAYERS)]
        self.latent = [torch.full((NB, BS, R + DR), float("nan"), device="cuda").bfloat16() for _ in range(LAYERS)]
        self.sets = pkv.PoolSet(self.kv), pkv.LatentPoolSet(self.latent)
        self.rope = pkv.make_rope(10000.0 ** (-2.0 * np.arange(DR // 2) / DR), interleaved=True)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = pkv.alloc_workspace(max(pkv.tree_workspace_size(3, HQ, HKV, D, BS, 64, 1024),
                                          pkv.latent_workspace_size(3, H, R, DR, BS, 64, 1024)), "cuda")
        self.n = np.zeros(3, dtype=np.int64)                      # committed tokens
        # what every committed token's row is: [row][layer] lists of (k, v, latent row)
        self.rows = [[[] for _ in range(LAYERS)] for _ in range(3)]

    def tables(self, lens):
        rows = []
        for r, L in enumerate(lens):
            self.alloc.reserve(self.req[r], int(L))
            rows.append(self.alloc.table(self.req[r]))
        t = np.full((3, max(len(x) for x in rows)), -1, dtype=np.int32)
        for r, x in enumerate(rows):
            t[r, :len(x)] = x
        return t

    def append(self, counts, positions):
        """counts[r] new tokens behind each row's committed ones; their rows as the caches hold them."""
        pkv, lens = self.pkv, self.n + counts
        t = self.tables(lens)
        at = [np.arange(n, n + c) for n, c in zip(self.n, counts)]
        slots = to(np.concatenate([t[r, p // BS] * BS + p % BS for r, p in enumerate(at)]).astype(np.int32))
        T, pos = int(counts.sum()), to(np.concatenate(positions).astype(np.int32))
        new = [[[] for _ in range(LAYERS)] for _ in range(3)]
        cut = np.concatenate([[0], np.cumsum(counts)])
        for layer in range(LAYERS):
            k, v, c, kr = [as_type(self.rng.randn(T, *s), "bf16").cuda() for s in ((HKV, D), (HKV, D), (R,), (DR,))]
            pkv.paged_kv_append(*self.kv[layer], slots, k, v, status=self.status,
                                **(dict(k_scale=KS, v_scale=VS) if self.kind == "fp8" else {}))
            pkv.paged_latent_append(self.latent[layer], slots, c, kr, pos, self.rope, status=self.status)
            held = f64(self.latent[layer].view(-1, R + DR)[slots.long()])
            assert np.array_equal(held[:, :R], f64(c))
            if self.kind == "fp8":
                q8 = lambda x, s: f64((x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn)) * s  # noqa: E731
                k, v = q8(k, KS), q8(v, VS)
            else:
                k, v = f64(k), f64(v)
            for r in range(3):
                s = slice(cut[r], cut[r + 1])
                new[r][layer] = list(zip(k[s], v[s], held[s]))
        return t, lens, new

    def prompt(self, counts):
        counts = np.array(counts)
        _, self.n, new = self.append(counts, [np.arange(c) for c in counts])
        self.rows = new

    def step(self, nodes):
        pkv, nodes = self.pkv, np.array(nodes)
        cu = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        up = [random_tree(self.rng, c) for c in nodes]
        masks = pkv.tree_masks_host(np.concatenate(up), cu)
        depth = [np.array([bin(int(m) & (1 << 64) - 1).count("1") - 1 for m in masks[a:b]], dtype=np.int64)
                 for a, b in zip(cu, cu[1:])]
        t, lens, new = self.append(nodes, [n + d for n, d in zip(self.n, depth)])
        d_t, d_L, d_cu, d_m = to(t), to(lens.astype(np.int32)), to(cu), to(masks)
        max_q, max_len = int(nodes.max()), int(lens.max())
        for layer in range(LAYERS):
            q = as_type(self.rng.randn(int(cu[-1]), HQ, D), "bf16")
            lq = as_type(self.rng.randn(int(cu[-1]), H, R + DR) * (2.0 / (R + DR)) ** 0.25, "bf16")
            kp, vp = self.kv[layer]
            out = pkv.paged_tree_attention(q.cuda(), d_cu, d_m, kp, vp, d_t, d_L, max_q, 0, D ** -0.5, workspace=self.ws,
                                           max_seq_len=max_len, status=self.status,
                                           **(dict(k_scale=KS, v_scale=VS) if self.kind == "fp8" else {}))
            lout = pkv.paged_latent_attention(lq.cuda(), self.latent[layer], R, d_t, d_L, 0.125, cu_q_lens=d_cu, max_q_len=max_q,
                                              tree_masks=d_m, workspace=self.ws, max_seq_len=max_len, status=self.status)
            for r in range(3):
                a, b = cu[r], cu[r + 1]
                held = self.rows[r][layer] + new[r][layer]
                k, v, lat = [np.array([x[i] for x in held]) for i in range(3)]
                ok = seen(int(lens[r]), int(nodes[r]), masks[a:b])
                for h in range(0, HQ, 5):
                    g = h * HKV // HQ
                    ref, mag, A = attend(f64(q)[a:b, h], k[:, g], v[:, g], ok, D ** -0.5)
                    check(out[a:b, h], ref, mag, A, D, self.kind, torch.bfloat16, f"layer {layer} row {r} head {h}")
                    ref, mag, A = attend(f64(lq)[a:b, h], lat, lat[:, :R], ok, 0.125)
                    check(lout[a:b, h], ref, mag, A, R + DR, "bf16 weights", torch.bfloat16, f"latent {layer} {r} {h}")
        # the accepted paths: from a root down, one of the children each time
        paths = []
        for u in up:
            walk, node = [], -1
            while len(walk) < self.rng.randint(0, 12):
                kids = [i for i, p in enumerate(u) if p == node]
                if not kids:
                    break
                node = kids[self.rng.randint(len(kids))]
                walk.append(node)
            paths.append(walk)
        path = np.full((3, max_q), -1, dtype=np.int32)
        for r, w in enumerate(paths):
            path[r, :len(w)] = w
        count = to(np.array([len(w) for w in paths], dtype=np.int32))
        lengths = [pkv.paged_tree_commit(s, d_t, d_L, d_cu, to(path), count, status=self.status) for s in self.sets]
        assert torch.equal(*lengths) and int(self.status.item()) == 0
        self.n = np.array(lengths[0].tolist())
        for r, w in enumerate(paths):
            for layer in range(LAYERS):
                self.rows[r][layer] += [new[r][layer][i] for i in w]
            assert self.n[r] == len(self.rows[r][0])
            assert self.alloc.truncate(self.req[r], int(self.n[r])) is None   # nobody shares these pages
            # the latent cache holds exactly the accepted rows (the K/V one is read by the next step)
            pages = self.alloc.table(self.req[r])
            p = np.arange(self.n[r])
            for layer in range(LAYERS):
                got = f64(self.latent[layer].view(-1, R + DR)[to((pages[p // BS] * BS + p % BS).astype(np.int64))])
                assert np.array_equal(got, np.array([x[2] for x in self.rows[r][layer]]).reshape(got.shape))


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_speculative_steps(pkv, kind):
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        server = Server(pkv, kind, 11)
        server.prompt([5, 33, 16])
        for nodes in ([3, 16, 4], [40, 1, 9], [4, 4, 4], [64, 17, 2], [1, 1, 1]):
            server.step(nodes)
    assert server.n.min() >= 5
