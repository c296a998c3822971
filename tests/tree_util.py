"""Paged inputs and 64-bit forms for drafted trees and latent caches.

Bounds: an output is off by its rounding (half a step of its type), and by the
errors of its weights.  A score of W products is off by at most
W 2^-23 sum |q k| scale (fp32 sums, each step rounded or cut), a weight then
relatively by twice that (its own and the normaliser's), plus the weight's own
rounding and the exponential's (`weight`): 2^-16 where weights are carried in two
bf16 terms or fp32, 2^-10 where they are one f16 term (2^-11, twice).

Weights that are one bf16 term, with the sum taken over the rounded ones ("bf16
weights"): with p the exact weights, L their sum, |d| <= e = 2^-8 each one's rounding
and d' = sum p d / L, so |d'| <= e, the output differs by
    |(sum p (1 + d) v) / (L (1 + d')) - sum p v / L| = |sum p d v - d' sum p v| / (L (1 + d'))
                                                    <= 2 e / (1 - e) * sum p |v| / L,
which is 2^-7 (1 + 2^-8 + ..) <= 2^-7 + 2^-14 - 2^-16, leaving 2^-16 for the exponential."""
from __future__ import annotations

import numpy as np
import torch

BS = 16
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
WEIGHT = {"f32": 2.0 ** -16, "bf16": 2.0 ** -16, "fp8": 2.0 ** -10, "bf16 weights": 2.0 ** -7 + 2.0 ** -14}


def random_tree(rng, n, chain=0.4):
    return np.array([i - 1 if rng.rand() < chain else rng.randint(-1, i) for i in range(n)], dtype=np.int32)


def tables_for(rng, lens, lo=None, extra=3, bs=BS):
    """Shuffled pages for rows of these lengths (-1 before position lo), with unused pages among them."""
    width = max(1, max(-(-int(n) // bs) for n in lens))
    t = np.full((len(lens), width), -1, dtype=np.int32)
    held = [(r, b) for r, n in enumerate(lens) for b in range((int(lo[r]) // bs) if lo is not None else 0, -(-int(n) // bs))]
    nb = len(held) + extra
    for (r, b), x in zip(held, rng.permutation(nb)):
        t[r, b] = x
    return t, nb


def fill(pool, tables, r, L, rows, bs=BS):
    """rows [L, ...] into row r's pages of a [nb, bs, ...] pool (positions whose page is -1 left out)."""
    for p in range(L):
        b = tables[r, p // bs]
        if b >= 0:
            pool[b, p % bs] = rows[p]


def seen(L, C, masks=None, window=0):
    """[C, L] truth values: what each of the last C positions' queries attends."""
    n = L - C
    out = np.zeros((C, L), dtype=bool)
    for i in range(C):
        mine = [j for j in range(i + 1) if masks is None or (int(masks[i]) >> j) & 1]
        at = n + (i if masks is None else max(0, len(mine) - 1))
        out[i, max(0, at - window + 1) if window else 0:n] = True
        out[i, [n + j for j in mine]] = True
        if masks is None and window:
            out[i, :max(0, at - window + 1)] = False
    return out


def attend(q, k, v, ok, scale):
    """64-bit attention of q [C, D] over k [L, D], v [L, Dv] where ok [C, L]: out, sum p |v|, max sum |q k| scale."""
    s = (q @ k.T) * scale
    A = float((np.abs(q) @ np.abs(k).T).max() * abs(scale)) if k.size and q.size else 0.0
    s = np.where(ok, s, -np.inf)
    m = np.max(s, axis=1, keepdims=True, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(m), m, 0.0))
    l = e.sum(1, keepdims=True)
    p = np.divide(e, l, out=np.zeros_like(e), where=l > 0)
    return p @ v, p @ np.abs(v), A


def check(got, ref, mag, A, W, kind, dtype, what=""):
    """got [.., Dv] against the 64-bit ref within the bound above."""
    got = got.detach().float().cpu().numpy().astype(np.float64)
    bound = HALF[dtype] * np.abs(ref) + (2 * W * 2.0 ** -23 * A + WEIGHT[kind]) * mag + 1e-30
    err = np.abs(got - ref)
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = float((err / bound).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.2f} of the bound at {np.unravel_index((err / bound).argmax(), err.shape)}"


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def as_type(a, kind):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)) if kind == "f32" else bf16(a)


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)
