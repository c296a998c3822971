"""The division-free E4M3 quotient on float32 inputs (the rotary append quantises
rotated rows before any rounding to bf16).

q0 = RN(x r), r = RN(1 / s), is off the quotient by up to 1.5 ulp (half an ulp of
its own, up to one from r's), so that e = x - s q0 may need a 25th bit and q1 =
RN(q0 + e r) is the rounding of a number off x / s by up to 1.5 ulp (2^-24 of e's
rounding + 2^-24 of r's) = 3 * 2^-24 ulp.  That changes an E4M3 code only where
x / s lies that close to a boundary h = m +- half an ulp, m a midpoint between
codes: x = X 2^c, s = S 2^d with 24-bit X, S and m = M 2^j with 16 <= M <= 31 give
|x / s - h| = |D| / 2S ulp, D = X 2^24 (or 2^25) - S (M 2^20 +- 1) an integer, so
|D| < 2 * 2^24 * 3 * 2^-24 = 6.  Every such S (one per M, sign and D) is tried here,
out to |D| = 64; at m a power of two the lower boundary is a quarter ulp below.
"""
import numpy as np
import pytest

from test_fp8_quotient import _codes_division_free, _rn32_sum


def boundary_pairs():
    """(X, S) with |D| <= 64 at a boundary of some midpoint."""
    out = set()
    for M in range(16, 32):
        # the boundaries as odd integers H over a power of two 2^p
        for H, p in ((M * 2 ** 20 + 1, 24), (M * 2 ** 20 - 1, 24), (M * 2 ** 21 - 1, 25)):
            if p == 25 and M != 16:
                continue
            for k in (p, p + 1):                    # X 2^k near S H
                inv = pow(H, -1, 1 << k)
                for D in range(-64, 65):
                    S = -D * inv % (1 << k)
                    for S in (S, S - (1 << k)):
                        X, rest = divmod(S * H + D, 1 << k)
                        if (1 << 23) <= S < (1 << 24) and rest == 0 and (1 << 23) <= X < (1 << 24):
                            out.add((X, S, D))
    return sorted(out)


def codes(orc, x, s):
    """_codes_division_free for a scale per element."""
    r = np.float32(1.0) / s
    q0 = x * r
    e = (x.astype(np.float64) - s.astype(np.float64) * q0.astype(np.float64)).astype(np.float32)
    q1 = _rn32_sum(q0.astype(np.float64), e.astype(np.float64) * r.astype(np.float64))
    a = np.abs(q0)
    return orc.e4m3_encode(np.where((a >= np.float32(2.0 ** -11)) & (a <= np.float32(512.0)), q1, q0))


def test_inputs_at_the_boundaries(orc):
    pairs = boundary_pairs()
    assert {abs(d) for _, _, d in pairs} >= {1, 2, 3, 4, 5}
    x = np.array([p[0] for p in pairs], np.float32)
    s = np.array([p[1] for p in pairs], np.float32)
    for shift in range(-12, 12):                    # the quotient over the codes' range, and past both ends
        xs = x * np.float32(2.0 ** shift)
        for one in (s, s * np.float32(2.0 ** -30), s * np.float32(2.0 ** 40)):
            xx = xs * (one / s)                     # the same quotients at other scales
            for sign in (1, -1):
                q = (xx * np.float32(sign) / one).astype(np.float32)
                ref = orc.e4m3_encode(q)
                assert np.array_equal(codes(orc, xx * np.float32(sign), one), ref), (shift, sign)


@pytest.mark.parametrize("seed", range(4))
def test_inputs_near_scaled_midpoints(orc, seed):
    # random scales, every midpoint, the float32 values within 12 ulps of s * midpoint
    rng = np.random.default_rng(seed)
    grid = orc.e4m3_decode(np.arange(0x7F, dtype=np.uint8))         # 0 .. 448
    mids = ((grid[1:].astype(np.float64) + grid[:-1]) / 2)
    for _ in range(200):
        s = np.float32(2.0 ** rng.uniform(-20, 20))
        x = (mids * np.float64(s)).astype(np.float32)
        x = (x.view(np.int32)[:, None] + np.arange(-12, 13, dtype=np.int32)[None]).view(np.float32).reshape(-1)
        assert np.array_equal(_codes_division_free(orc, x, s), orc.e4m3_encode(x / s)), float(s)
