"""Rotary append (GPU): positions expanded over the axes and four axes, and the
E4M3 codes of rotated rows."""
import numpy as np
import pytest

import pkv_inputs as gen
from gpu_util import storage_bytes, to_torch
from test_gpu_rope import KS, Case, check, inv_freq, k_tile_bytes, run

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import block_paged_kv_gb300 as m
    return m


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("T", [1, 20, 1100])
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_one_row_of_positions_for_every_axis(pkv, dtype, T, axes):
    c = Case(800 + axes, dtype, T, 4, 2, 128, axes=axes, far=100000)
    c.pos = np.ascontiguousarray(np.broadcast_to(c.pos[:1], c.pos.shape))
    q, kp, vp, _ = run(pkv, c)                      # the rows written out
    c.pos = c.pos[:1]
    torch_pos = torch.from_numpy(c.pos).cuda().expand(axes, T)
    rope = pkv.make_rope(inv_freq(128), c.axis, num_axes=axes)
    kp2, vp2 = c.dev()
    q2 = pkv.paged_kv_append_rope(kp2, vp2, torch.from_numpy(c.slots).cuda(), to_torch(c.q, c.bits),
                                  to_torch(c.k, c.bits), to_torch(c.v, c.bits), torch_pos, rope, **c.scales)
    assert torch.equal(q, q2) and storage_bytes(kp) == storage_bytes(kp2) and storage_bytes(vp) == storage_bytes(vp2)


@pytest.mark.parametrize("dtype", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("T,interleaved", [(33, False), (33, True), (1030, False)])
def test_four_axes(pkv, orc, dtype, T, interleaved):
    check(pkv, orc, Case(810, dtype, T, 4, 2, 128, axes=4, rd=96, far=1 << 20), interleaved)


@pytest.mark.parametrize("D,rd", [(64, 64), (128, 128), (128, 48), (256, 256), (256, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T", [40, 1100])           # per token, and whole tiles
def test_fp8_codes_are_those_of_the_fp32_rotation(pkv, orc, D, rd, interleaved, T):
    # an f32 pool keeps the rotated rows before they are quantised: the FP8 pool's
    # K codes are the nearest E4M3 codes of the float32 quotients of those, bit for bit
    c = Case(820 + D, "fp8", T, 2, 3, D, rd=rd)
    _, kp, _, status = run(pkv, c, interleaved)
    assert status == 0
    f = Case(820 + D, "f32", T, 2, 3, D, rd=rd)
    f.slots, f.pos, f.axis = c.slots, c.pos, c.axis
    f.q, f.k, f.v = (gen.as_f32(x, "bf16") for x in (c.q, c.k, c.v))
    _, kf, _, _ = run(pkv, f, interleaved)
    s = c.slots
    rows = kf.cpu().numpy()[s // 16, :, s % 16]     # [T, hkv, D]
    want = orc.e4m3_encode((rows / np.float32(KS)).reshape(-1)).reshape(rows.shape)
    at = ((s // 16)[:, None, None], np.arange(3)[None, :, None], k_tile_bytes(D)[s % 16][:, None, :])
    assert np.array_equal(kp.cpu().numpy()[at], want)
