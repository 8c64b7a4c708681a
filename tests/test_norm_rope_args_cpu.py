"""Host-side checks of rq_norm_rope and its backward call: they answer before any device work.

Pointers passed below are never dereferenced: each call fails a check first, or has nothing to do."""
import ctypes

import pytest

from test_operator_args_cpu import ALIGN, INVALID, OK, P, UNSUPPORTED, rope_config, rq, tensor  # noqa: F401

WORKSPACE = 4


def norm_tensor(rq, weight=P, grad=4 * P, weight_grad=5 * P, **kw):
    return rq._norm_tensor(tensor(rq, **kw), weight, grad, weight_grad, 1536, 384, 128)


def call(rq, q, k=None, cfg=None, dtype=0, wdtype=0, batch=2, n=3, eps=1e-6, start=P, offsets=None, back=False,
         ws=8 * P, size=None):
    ref = lambda x: None if x is None else ctypes.byref(x)
    args = [ref(cfg if cfg is not None else rope_config(rq)), dtype, wdtype, batch, n, ref(q), ref(k), eps, start, offsets]
    if back:
        return rq.lib.rq_norm_rope_backward(*args, ws, rq.rq_norm_rope_workspace_bytes(128) if size is None else size, None)
    return rq.lib.rq_norm_rope(*args, None)


@pytest.mark.parametrize("back", [False, True])
def test_refusals(rq, back):
    t = lambda **kw: norm_tensor(rq, **kw)
    go = lambda q, **kw: call(rq, q, back=back, **kw)
    assert go(None) == INVALID
    assert go(t(), eps=-1e-9) == INVALID and go(t(), eps=float("nan")) == INVALID and go(t(), eps=1e39) == INVALID
    assert go(t(), dtype=3) == INVALID and go(t(), wdtype=-1) == INVALID
    assert go(t(), batch=-1) == INVALID and go(t(), n=-1) == INVALID
    assert go(t(heads=0)) == INVALID and go(t(in_=None)) == INVALID and go(t(out=None)) == INVALID
    assert go(t(in_=P + 1)) == ALIGN and go(t(in_=P + 2), dtype=2) == ALIGN
    assert go(t(weight=P + 2), wdtype=2) == ALIGN and go(t(), start=P + 2) == ALIGN
    assert go(t(out_head=64)) == INVALID          # two results in one place
    assert go(t(), cfg=rope_config(rq, head_dim=514)) == UNSUPPORTED
    assert go(t(), cfg=rope_config(rq, theta=1.0)) == INVALID
    assert go(t(), cfg=rope_config(rq, scaling=1, factor=1e-320)) == INVALID
    assert go(t(), batch=65536, n=65536) == UNSUPPORTED
    assert go(t(heads=1 << 30), batch=2) == UNSUPPORTED


def test_backward_refusals(rq):
    t = lambda **kw: norm_tensor(rq, **kw)
    assert call(rq, t(grad=None), back=True) == INVALID
    assert call(rq, t(grad=P + 1), back=True) == ALIGN and call(rq, t(weight_grad=P + 2), back=True) == ALIGN
    assert call(rq, t(), back=True, ws=None) == INVALID and call(rq, t(), back=True, ws=P + 8) == ALIGN
    assert call(rq, t(), back=True, size=rq.rq_norm_rope_workspace_bytes(128) - 1) == WORKSPACE


def test_nothing_to_do(rq):
    t = lambda **kw: norm_tensor(rq, **kw)
    assert call(rq, t(in_=None, out=None), batch=0) == OK and call(rq, t(in_=None, out=None), n=0) == OK
    assert call(rq, t(grad=None, weight_grad=None), n=0, back=True, ws=None) == OK
    assert rq.rq_norm_rope_workspace_bytes(1) == 0 and rq.rq_norm_rope_workspace_bytes(513) == 0
    assert rq.rq_norm_rope_workspace_bytes(512) > 0


def test_weight_gradients_in_one_place(rq):
    """The workspace is too small: what gets that far passed the check."""
    t = lambda at: norm_tensor(rq, weight_grad=at)
    go = lambda a, b: call(rq, t(a), t(b), back=True, size=0)
    assert go(5 * P, 5 * P) == INVALID and go(5 * P, 5 * P + 508) == INVALID and go(5 * P + 4, 5 * P) == INVALID
    assert go(5 * P, 5 * P + 512) == WORKSPACE and go(5 * P + 512, 5 * P) == WORKSPACE and go(5 * P, None) == WORKSPACE
