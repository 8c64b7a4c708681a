"""Host-side checks of the tree attention, page and rotary calls: they answer before any device work.

Pointers passed below are never dereferenced: each call fails a check first, or has nothing to do."""
import ctypes

import pytest

OK, INVALID, ALIGN, UNSUPPORTED = 0, 1, 2, 6
P = 0x10000


@pytest.fixture(scope="module")
def rq():
    import __graft_entry__
    __graft_entry__.build()
    import decode_attention_rq_gb300
    return decode_attention_rq_gb300


def cache_config(rq, **kw):
    base = dict(num_layers=24, loops_per_group=4, num_groups=1, num_heads=16, head_dim=128, group_size=32,
                max_batch=4, max_seq_len=8192, mode=0)
    base.update(kw)
    return rq.rq_config(**base)


def rope_config(rq, **kw):
    base = dict(head_dim=128, rotary_dim=128, interleaved=0, inverse=0, scaling=rq.RQ_ROPE_PLAIN, original_len=8192,
                theta=10000.0, factor=4.0, low_turns=1.0, high_turns=32.0, magnitude=0.0)
    base.update(kw)
    return rq.rq_rope_config(**base)


def tensor(rq, **kw):
    """A [2][4][3][128] tensor, contiguous."""
    base = dict(in_=P, out=2 * P, heads=4, in_row=1536, in_head=384, in_token=128, out_row=1536, out_head=384,
                out_token=128)
    base.update(kw)
    return rq._rope_tensor(**base)


def rope(rq, cfg, q, k=None, dtype=0, batch=2, n=3, start=P, offsets=None):
    ref = lambda x: None if x is None else ctypes.byref(x)
    return rq.lib.rq_rope(ref(cfg), dtype, batch, n, ref(q), ref(k), start, offsets, None)


@pytest.mark.parametrize("kw,status", [
    (dict(head_dim=1), UNSUPPORTED), (dict(head_dim=514), UNSUPPORTED), (dict(rotary_dim=0), UNSUPPORTED),
    (dict(rotary_dim=3), UNSUPPORTED), (dict(rotary_dim=130), UNSUPPORTED),
    (dict(head_dim=512, rotary_dim=258), UNSUPPORTED),
    (dict(theta=1.0), INVALID), (dict(theta=-5.0), INVALID), (dict(theta=float("inf")), INVALID),
    (dict(theta=float("nan")), INVALID), (dict(magnitude=float("nan")), INVALID), (dict(magnitude=1e39), INVALID),
    (dict(scaling=-1), INVALID), (dict(scaling=4), INVALID), (dict(scaling=1, factor=0.0), INVALID),
    (dict(scaling=2, factor=-1.0), INVALID), (dict(scaling=3, factor=float("inf")), INVALID),
    (dict(scaling=2, rotary_dim=2), INVALID), (dict(scaling=3, original_len=0), INVALID),
    (dict(scaling=3, low_turns=32.0), INVALID), (dict(scaling=3, high_turns=float("inf")), INVALID),
    (dict(scaling=1, factor=1e-320), INVALID),      # 1 / factor is not finite
    (dict(scaling=2, factor=1e-320), INVALID),      # theta becomes so small that a frequency is not
])
def test_rope_configurations(rq, kw, status):
    assert rope(rq, rope_config(rq, **kw), tensor(rq)) == status


def test_rope_arguments(rq):
    cfg, x = rope_config(rq), tensor(rq)
    assert rope(rq, None, x) == INVALID
    assert rope(rq, cfg, None, None) == INVALID
    assert rope(rq, cfg, x, dtype=3) == INVALID
    assert rope(rq, cfg, x, dtype=-1) == INVALID
    assert rope(rq, cfg, x, batch=-1) == INVALID
    assert rope(rq, cfg, x, n=-1) == INVALID
    assert rope(rq, cfg, tensor(rq, heads=0)) == INVALID
    assert rope(rq, cfg, tensor(rq, in_=None)) == INVALID
    assert rope(rq, cfg, x, tensor(rq, out=None)) == INVALID
    assert rope(rq, cfg, tensor(rq, in_=P + 1)) == ALIGN
    assert rope(rq, cfg, tensor(rq, out=P + 2), dtype=2) == ALIGN
    assert rope(rq, cfg, x, start=P + 2) == ALIGN
    assert rope(rq, cfg, x, offsets=P + 1) == ALIGN
    assert rope(rq, cfg, tensor(rq, heads=1 << 30)) == UNSUPPORTED
    for stride in ("out_row", "out_head", "out_token"):     # two results in one place
        assert rope(rq, cfg, tensor(rq, **{stride: 0})) == INVALID
        assert rope(rq, cfg, x, tensor(rq, **{stride: 0})) == INVALID
    # nothing to do: no pointer is needed, nothing is launched
    assert rope(rq, cfg, tensor(rq, in_=None, out=None), batch=0) == OK
    assert rope(rq, cfg, tensor(rq, in_=None, out=None), n=0, start=None) == OK


def test_tree_workspace(rq):
    size = rq.rq_tree_workspace_bytes
    cfg = cache_config(rq)
    for batch, nodes in ((0, 4), (-1, 4), (4, 0), (4, -1), (4, rq.RQ_MAX_TREE_NODES + 1)):
        assert size(cfg, batch, nodes) == 0
    assert size(cfg, 4, rq.RQ_MAX_TREE_NODES) >= size(cfg, 4, 1) > 0
    for kw in (dict(head_dim=64), dict(num_heads=0), dict(mode=8), dict(num_query_heads=17)):
        assert size(cache_config(rq, **kw), 4, 4) == 0
    assert rq.lib.rq_tree_workspace_bytes(None, 4, 4) == 0
    assert rq.RQ_MAX_TREE_NODES == 256


def test_tree_and_page_calls_without_a_cache(rq):
    lib = rq.lib
    assert lib.rq_tree_attention(None, 0, 0, 0, 1, 4, P, P, P, P, P, P, 0.1, P, P, 1 << 30, None) == INVALID
    assert lib.rq_pages_copy(None, 1, P, P, None, None) == INVALID
    assert lib.rq_pages_fork(None, 1, P, P, P, None, None) == INVALID
    assert lib.rq_pages_reserve(None, 1, P, 1, P, None, P, 1 << 30, None) == INVALID
    assert lib.rq_pages_free(None, 1, P, None, P, None, None) == INVALID
    assert lib.rq_pages_compact(None, P, P, None, P, 1 << 30, None) == INVALID


def test_page_workspace(rq):
    size = rq.rq_pages_workspace_bytes
    assert size(cache_config(rq), 0) == 0
    assert size(cache_config(rq), -5) == 0
    assert size(cache_config(rq, group_size=8), 100) == 0
    assert rq.lib.rq_pages_workspace_bytes(None, 100) == 0
    assert size(cache_config(rq), 100) >= 6 * 400
