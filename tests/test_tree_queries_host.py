"""paged_tree_attention_queries on the CPU: refusals before any launch."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def pkv():
    import block_paged_kv_gb300 as m
    return m


def test_refused_before_launch(pkv):
    pool = pkv._Pool(16, 16, 4, 16, 2, 128, pkv.PKV_BF16, 0.0, 0.0)

    def call(n, masks=16, max_q=4, q=16, window=0):
        return pkv._lib.paged_tree_attention_queries(q, n, 16, masks, 4, ctypes.byref(pool), 16, 8, 16, 1, max_q, 64, window,
                                                     0.1, 16, 256, 0, None, None)

    bad = pkv.PKV_ERR_INVALID_ARG
    assert call(-1) == bad and call(4, max_q=65) == bad and call(4, masks=None) == bad and call(4, q=8) == bad
    assert call(0, max_q=-1) == bad and call(0, max_q=65) == bad
    assert call(4, window=3) == pkv.PKV_ERR_UNSUPPORTED
    assert call(0) == pkv.PKV_OK and call(0, masks=None) == pkv.PKV_OK     # nothing to launch
    assert call(4) == pkv.PKV_ERR_WORKSPACE
