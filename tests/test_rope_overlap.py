"""rq_rope refuses strides that put two results of a tensor in one place, and no others (host-side check).

Every call below fails a later check if it passes this one: start is misaligned, so nothing is launched."""
import ctypes
import itertools
import random

import pytest

INVALID, ALIGN = 1, 2
P = 0x10000


@pytest.fixture(scope="module")
def rq():
    import __graft_entry__
    __graft_entry__.build()
    import decode_attention_rq_gb300
    return decode_attention_rq_gb300


def status(rq, d, batch, heads, n, row, head, token, as_k=False):
    cfg = rq.rq_rope_config(head_dim=d, rotary_dim=2, theta=10000.0)
    x = rq._rope_tensor(P, 2 * P, heads, d * heads * n, d * n, d, row, head, token)
    other = rq._rope_tensor(P, 2 * P, 1, d * n, d * n, d, d * n, d * n, d)
    q, k = (other, x) if as_k else (x, None)
    return rq.lib.rq_rope(ctypes.byref(cfg), 0, batch, n, ctypes.byref(q), None if k is None else ctypes.byref(k), P + 2,
                          None, None)


def overlaps(d, sizes, strides):
    """By the elements themselves."""
    seen = set()
    for at in itertools.product(*(range(s) for s in sizes)):
        first = sum(a * b for a, b in zip(at, strides))
        for c in range(d):
            if first + c in seen:
                return True
            seen.add(first + c)
    return False


@pytest.mark.parametrize("name,sizes,strides,bad", [
    ("contiguous", (2, 4, 3), (1536, 384, 128), False),
    ("token-major", (2, 4, 3), (1536, 128, 512), False),
    ("a view of a wider projection", (2, 4, 3), (4608, 128, 1536), False),
    ("rows innermost", (2, 4, 3), (128, 256, 1024), False),
    ("backwards", (2, 4, 3), (1536, -384, -128), False),
    ("a token inside the one before", (2, 4, 3), (1536, 384, 64), True),
    ("one channel short", (2, 4, 3), (1536, 384, 127), True),
    ("heads inside the tokens of the one before", (1, 4, 3), (0, 256, 128), True),
    ("rows inside the heads of the one before", (2, 4, 3), (1152, 384, 128), True),
    ("rows inside, backwards", (2, 4, 3), (-1152, 384, 128), True),
    ("heads between the tokens", (1, 2, 3), (0, 384, 256), False),
    ("heads and tokens meet", (1, 3, 4), (0, 384, 256), True),
    ("axes of one need no stride", (1, 1, 1), (0, 0, 0), False),
    ("axes of one may have any", (1, 1, 3), (1, -7, 128), False),
    ("one axis alone", (1, 1, 3), (0, 0, 100), True),
    ("large", (4, 1 << 20, 1 << 9), (1 << 36, 1 << 16, 128), False),
    ("large, one short", (4, 1 << 20, 1 << 9), (1 << 36, (1 << 16) - 1, 128), True),
    ("the largest", (2, 2, 2), ((1 << 63) - 1, -(1 << 62), 128), False),
    ("the largest, which differ by one", (2, 2, 2), ((1 << 63) - 1, -(1 << 63), 128), True),
])
def test_layouts(rq, name, sizes, strides, bad):
    for as_k in (False, True):
        assert status(rq, 128, *sizes, *strides, as_k=as_k) == (INVALID if bad else ALIGN), name


def test_random_layouts_against_their_elements(rq):
    rng = random.Random(0)
    count = [0, 0]
    for _ in range(6000):
        d = rng.choice([2, 3, 5, 8])
        sizes = [rng.choice([1, 2, 3, 4, 5]) for _ in range(3)]
        strides = [rng.choice([-1, 1]) * rng.randrange(1, 10 * d) for _ in range(3)]
        if rng.random() < 0.5:      # multiples of the head, an odd rest now and then: many that interlock
            strides = [rng.choice([-1, 1]) * rng.randrange(1, 14) * d + (rng.random() < 0.1) for _ in range(3)]
        bad = overlaps(d, sizes, strides)
        if any(n > 1 and s == 0 for n, s in zip(sizes, strides)):
            bad = True
        count[bad] += 1
        assert status(rq, d, *sizes, *strides) == (INVALID if bad else ALIGN), (d, sizes, strides)
    assert min(count) > 600


def test_nothing_to_do_is_not_refused(rq):
    cfg = rq.rq_rope_config(head_dim=128, rotary_dim=128, theta=10000.0)
    x = rq._rope_tensor(None, None, 4, 1536, 384, 128, 1536, 384, 64)
    assert rq.lib.rq_rope(ctypes.byref(cfg), 0, 2, 0, ctypes.byref(x), None, None, None, None) == 0
    assert rq.lib.rq_rope(ctypes.byref(cfg), 0, 0, 3, ctypes.byref(x), None, None, None, None) == 0
