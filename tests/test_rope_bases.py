"""rq_rope refuses a stretched base that leaves float64: its frequencies would be zero (host-side check)."""
import ctypes

import pytest

INVALID = 1
P = 0x10000


@pytest.mark.parametrize("r,theta,factor", [(4, 10000.0, 1e153), (128, 1e10, 1e300), (4, 1e308, 2.0)])
def test_bases_out_of_range(r, theta, factor):
    import __graft_entry__
    __graft_entry__.build()
    import decode_attention_rq_gb300 as rq
    cfg = rq.rq_rope_config(head_dim=128, rotary_dim=r, scaling=rq.RQ_ROPE_BASE, theta=theta, factor=factor)
    x = rq._rope_tensor(P, 2 * P, 4, 1536, 384, 128, 1536, 384, 128)
    assert rq.lib.rq_rope(ctypes.byref(cfg), 0, 2, 3, ctypes.byref(x), None, P, None, None) == INVALID
